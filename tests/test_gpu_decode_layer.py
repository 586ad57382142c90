"""The decode layer's operators as they are used together: one decoder layer of ternary
projections, several tokens in turn, eagerly and as a replayed CUDA graph whose positions,
slots and lengths advance on the device.  Each operator is held, on the values that really
reached it, to its own float64 form."""
import numpy as np
import pytest

import oracle
from tests import layer_ref as ref
from tests.gpu_util import Problem, to_numpy_f16
from tests.test_gpu_epilogue import check as check_epilogue
from tests.test_gpu_parity import swiglu_ok

pytestmark = pytest.mark.gpu

HQ, HKV, D, PAGE, F = 4, 2, 64, 16, 512
DIM = HQ * D


@pytest.fixture(scope="module")
def bz():
    import torch
    from ternary_weight_02_b200 import bonsai
    assert bonsai.bonsai_check_device() == bonsai.BONSAI_OK
    torch.cuda.init()
    return bonsai


class Layer:
    """Weights, cache and buffers of one decoder layer for B sequences with given lengths."""

    def __init__(self, bz, fmt, B, kv, lengths, new_tokens, seed=0):
        import torch
        self.bz, self.fmt, self.B, self.kv = bz, fmt, B, kv
        rng = np.random.default_rng(seed)
        shapes = {"qkv": ((HQ + 2 * HKV) * D, DIM), "o": (DIM, DIM), "gate_up": (2 * F, DIM), "down": (DIM, F)}
        self.w = {k: Problem(0, N, K, fmt, seed=seed + i) for i, (k, (N, K)) in enumerate(shapes.items())}
        self.dev = {k: p.device()[1:] for k, p in self.w.items()}
        self.bias = rng.normal(0, 1, shapes["qkv"][0]).astype(np.float16)
        self.bias_d = self.up(self.bias)
        self.freqs = bz.bonsai_rope_frequencies(D, 1e4)[0].cuda()
        width = -(-(max(lengths) + new_tokens) // PAGE)
        self.table = torch.from_numpy(rng.permutation(B * width).astype(np.int32).reshape(B, width)).cuda()
        kind = torch.float8_e4m3fn if kv else torch.float16
        one = lambda lo, hi: torch.from_numpy(rng.uniform(lo, hi, HKV).astype(np.float32)).cuda()  # noqa: E731
        self.scales = [one(0.02, 0.04), one(0.1, 0.2)] if kv else [None, None]
        past = [torch.from_numpy(rng.normal(0, 1, (B * width, HKV, PAGE, D)).astype(np.float32)).cuda() for _ in range(2)]
        self.pools = [(p / s[:, None, None] if kv else p).to(kind) for p, s in zip(past, self.scales)]
        self.start = torch.tensor(lengths, dtype=torch.int32, device="cuda")
        self.lengths, self.positions = self.start.clone(), self.start.clone()
        self.slots = torch.zeros(B, dtype=torch.int64, device="cuda")
        self.x0 = self.up(rng.normal(0, 1, (B, DIM)).astype(np.float16))
        f16 = dict(dtype=torch.float16, device="cuda")
        self.x, self.x1 = self.x0.clone(), torch.empty((B, DIM), **f16)
        self.qkv, self.q, self.att, self.h = (torch.empty((B, n), **f16) for n in (shapes["qkv"][0], DIM, DIM, F))

    @staticmethod
    def up(a):
        import torch
        return torch.from_numpy(a.view(np.int16)).cuda().view(torch.float16)

    def reset(self):
        self.x.copy_(self.x0)
        self.lengths.copy_(self.start)

    def step(self):
        """One token per sequence: x becomes the layer's output."""
        import torch
        bz, B, N = self.bz, self.B, (HQ + 2 * HKV) * D
        self.positions.copy_(self.lengths)
        page = torch.gather(self.table, 1, (self.positions // PAGE).long()[:, None])[:, 0].long()
        self.slots.copy_(page * PAGE + self.positions % PAGE)
        self.lengths.add_(1)
        bz.bonsai_ternary_linear_epilogue(self.x, *self.dev["qkv"], self.bias_d, None, self.qkv, B, N, DIM, self.fmt)
        bz.bonsai_rope_append(self.qkv, self.q, *self.pools, *self.scales, self.freqs, self.positions, self.slots, B, HQ, D)
        bz.bonsai_paged_attention(self.q, *self.pools, *self.scales, self.table, self.lengths, self.att, B, HQ)
        bz.bonsai_ternary_linear_epilogue(self.att, *self.dev["o"], None, self.x, self.x1, B, DIM, DIM, self.fmt)
        bz.bonsai_ternary_linear_swiglu(self.x1, *self.dev["gate_up"], self.h, B, F, DIM, self.fmt)
        bz.bonsai_ternary_linear_epilogue(self.h, *self.dev["down"], None, self.x1, self.x, B, DIM, F, self.fmt)

    def product(self, name, x):
        p = self.w[name]
        return oracle.ternary_linear(x, p.oracle_packed(), p.scales, p.N, p.K, self.fmt)

    def check_step(self, x_in):
        """Every operator of the step just made, on the values that reached it."""
        import torch
        B = self.B
        half = lambda t: t.cpu().numpy()  # noqa: E731
        qkv = half(self.qkv)
        check_epilogue(qkv.astype(np.float64), self.product("qkv", x_in), self.bias, None, 0)
        heads = qkv.reshape(B, -1, D).astype(np.float64)
        rot, slack = ref.rope(heads[:, : HQ + HKV], half(self.positions), half(self.freqs), D, 0, 1.0)
        bound = ref.f16_bound(rot, slack)
        q = half(self.q).reshape(B, HQ, D)
        assert (np.abs(q.astype(np.float64) - rot[:, :HQ]) <= bound[:, :HQ]).all()
        # the cache as it is now, sequence by sequence
        bits = torch.uint8 if self.kv else torch.int16
        table, n = half(self.table), half(self.lengths)
        entries = []
        for pool, s in zip(self.pools, self.scales):
            raw = pool.view(bits).cpu().numpy()
            vals = ref.e4m3_values(raw) * half(s)[None, :, None, None].astype(np.float64) if self.kv \
                else raw.view(np.float16).astype(np.float64)
            entries.append([vals[table[b]].transpose(0, 2, 1, 3).reshape(-1, HKV, D)[: n[b]] for b in range(B)])
        k_new = np.stack([entries[0][b][-1] for b in range(B)])
        if self.kv:
            s = half(self.scales[0])[None, :, None].astype(np.float64)
            u = np.clip(rot[:, HQ:] / s, -448, 448)
            assert (np.abs(k_new / s - u) <= ref.e4m3_bound(u, slack[:, HQ:] / s) + 2.0 ** -50 * np.abs(u)).all()
        else:
            assert (np.abs(k_new - rot[:, HQ:]) <= bound[:, HQ:]).all()
        want, _, tol, _ = ref.attention(q.astype(np.float64), *entries, n, 0, D ** -0.5)
        att = half(self.att)
        assert (np.abs(att.reshape(B, HQ, D).astype(np.float64) - want) <= tol).all()
        x1 = half(self.x1)
        check_epilogue(x1.astype(np.float64), self.product("o", att), None, x_in, 0)
        ok, rel, worst = swiglu_ok(to_numpy_f16(self.h), self.product("gate_up", x1))
        assert ok, (rel, worst)
        check_epilogue(to_numpy_f16(self.x), self.product("down", half(self.h)), None, x1, 0)


@pytest.mark.parametrize("fmt,B,kv", [(oracle.FMT_PQ2_0, 1, 0), (oracle.FMT_PQ2_0, 3, 1), (oracle.FMT_PTQ1_0, 1, 1),
                                      (oracle.FMT_Q1_0, 5, 0), (oracle.FMT_PQ2_0_G64, 20, 0)])
def test_decode_layer_steps(bz, fmt, B, kv):
    import torch
    lengths = [(37 * i + 13) % 90 for i in range(B)]
    layer = Layer(bz, fmt, B, kv, lengths, 4, seed=B)
    for _ in range(4):
        x_in = layer.x.cpu().numpy()
        layer.step()
        torch.cuda.synchronize()
        layer.check_step(x_in)
    assert bz.bonsai_device_status(clear=True) == 0


@pytest.mark.parametrize("B,kv", [(1, 0), (4, 1)])
def test_decode_layer_as_a_replayed_graph(bz, B, kv):
    """A captured step, replayed, writes the bits that eager steps write, token after token."""
    import torch
    layer = Layer(bz, oracle.FMT_PQ2_0, B, kv, [29 + i for i in range(B)], 6, seed=7)
    bz.bonsai_reserve(B, 2 * F, F)
    pools = [p.clone() for p in layer.pools]
    eager = []
    for _ in range(5):
        layer.step()
        eager.append(layer.x.clone())
    end = [p.clone() for p in layer.pools]
    layer.reset()
    for p, c in zip(layer.pools, pools):
        p.copy_(c)
    torch.cuda.synchronize()
    s, g = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        layer.step()
    layer.reset()
    for want in eager:
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(layer.x, want)
    for p, c in zip(layer.pools, end):
        assert torch.equal(p.view(torch.uint8), c.view(torch.uint8))
    del g


def test_calls_on_two_streams_in_turn(bz):
    """Calls that share the workspace, on two streams ordered by events: same bits as on one."""
    import torch
    layer = Layer(bz, oracle.FMT_PQ2_0, 2, 0, [50, 3], 3, seed=9)
    layer.step()
    want = layer.x.clone()
    layer.reset()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        layer.step()
    torch.cuda.current_stream().wait_stream(s)
    assert torch.equal(layer.x, want)
