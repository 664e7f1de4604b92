"""Cross attention to an encoder's states on the GPU: forward and gradients against the float64
definition, element by element, with bounds derived from the roundings the kernels make (bf16:
2^-8 of a value for a rounding to nearest; sums, statistics and scores are fp32)."""
import numpy as np
import pytest
import torch

import oracle
from mla_latent_kv_attn_b200 import api, rollout

pytestmark = pytest.mark.gpu

BF16 = 2.0 ** -8
# The tensor-core kernels round P to bf16; ex2.approx is off by 2^-22, and so, at most, is each of the
# two products behind a dS.
P_REL = BF16 + 2.0 ** -20


class Case:
    """Inputs (rounded to T) and zero-filled outputs of one call."""

    def __init__(self, B, n_q, n_kv, H, Hkv, d, lens=None, dtype="bf16", path=api.MLA_PATH_AUTO,
                 scale=None, std=1.0, seed=0, wide=False):
        self.cc = api.make_cross_config(batch=B, n_heads=H, n_kv_heads=Hkv, d_head=d, n_q=n_q,
                                        n_kv=n_kv, softmax_scale=scale, dtype=dtype,
                                        kernel_path=path)
        self.dt = torch.float32 if dtype == "fp32" else torch.bfloat16
        g = torch.Generator(device="cuda").manual_seed(seed)
        new = lambda *shape: (torch.randn(shape, generator=g, device="cuda") * std).to(self.dt)
        if wide:      # parts of the rows of wider projections
            self.q = new(B, n_q, H * d + 32)[..., 16:16 + H * d].unflatten(-1, (H, d))
            kv = new(B, n_kv, 2, Hkv, d)
            self.k, self.v = kv[:, :, 0], kv[:, :, 1]
        else:
            self.q, self.k, self.v = new(B, n_q, H, d), new(B, n_kv, Hkv, d), new(B, n_kv, Hkv, d)
        self.g = new(B, n_q, H, d)
        self.lens = lens
        self.kv_len = None if lens is None else torch.tensor(lens, device="cuda",
                                                             dtype=torch.int32)
        self.out = torch.full((B, n_q, H, d), 7.0, device="cuda", dtype=self.dt)
        self.lse = torch.full((B, H, n_q), 7.0, device="cuda")
        self.status = torch.zeros(1, device="cuda", dtype=torch.int32)
        need = api.mla_cross_attention_bwd_workspace_bytes(self.cc)
        self.ws = torch.full((need,), 0xFF, device="cuda", dtype=torch.uint8)      # NaN
        self.grads = [torch.full(s, 7.0, device="cuda", dtype=self.dt)
                      for s in ((B, n_q, H, d), (B, n_kv, Hkv, d), (B, n_kv, Hkv, d))]

    def fwd(self, stream=None, lse=True):
        api.mla_cross_attention_fwd(self.cc, self.q, self.k, self.v, self.out,
                                    lse=self.lse if lse else None, kv_len=self.kv_len,
                                    dev_status=self.status, stream=stream)

    def bwd(self, stream=None):
        api.mla_cross_attention_bwd(self.cc, self.q, self.k, self.v, self.out, self.lse, self.g,
                                    *self.grads, self.ws, kv_len=self.kv_len,
                                    dev_status=self.status, stream=stream)

    def check(self, backward=True):
        lens = [self.cc.n_kv] * self.cc.batch if self.lens is None else self.lens
        np64 = lambda t: t.double().cpu().numpy()
        fp32 = self.dt == torch.float32
        r, p_rel = (2.0 ** -24, 2.0 ** -22) if fp32 else (BF16, P_REL)
        args = (np64(self.q), np64(self.k), np64(self.v), lens, self.cc.softmax_scale)
        out, lse, e_out, e_lse = oracle.cross_attention(*args, p_rel=p_rel)
        assert int(self.status) == 0
        close("out", np64(self.out), out, e_out * (1 + r) + r * np.abs(out))
        got = np64(self.lse)
        assert np.array_equal(np.isneginf(got), np.isneginf(lse))
        ok = np.isfinite(lse)
        close("lse", got[ok], lse[ok], e_lse[ok] + 2.0 ** -22)
        if not backward:
            return
        # dS is computed from fp32 P and rounded once; P_REL covers P as an operand of dV
        want, err = oracle.cross_attention_backward(
            *args, np64(self.g), p_rel=p_rel, o_rel=r, ds_rel=2.0 ** -21 if fp32 else P_REL,
            fwd_rel=p_rel)
        for name, t, w, e in zip(("d_q", "d_k", "d_v"), self.grads, want, err):
            close(name, np64(t), w, e * (1 + r) + r * np.abs(w))


def close(name, got, want, bound):
    """Every element within its bound, a value of zero up to the smallest bf16 normal."""
    bad = np.abs(got - want) > bound + 2.0 ** -120
    assert np.isfinite(got).all(), name
    assert not bad.any(), (name, int(bad.sum()), float(np.abs(got - want).max()),
                           float((np.abs(got - want) / (bound + 2.0 ** -120)).max()))


SHAPES = [
    # B, n_q, n_kv, H, Hkv, d, lens
    (1, 1, 1, 1, 1, 128, None),
    (1, 1, 512, 3, 3, 128, None),
    (2, 5, 129, 4, 2, 64, [129, 77]),
    (2, 130, 64, 2, 1, 128, [64, 63]),
    (1, 257, 200, 4, 4, 128, [193]),
    (3, 70, 300, 6, 2, 64, [1, 0, 300]),
    (2, 200, 65, 12, 4, 128, [65, 1]),
    (1, 333, 1025, 4, 1, 64, [1025]),
    (4, 3, 40, 8, 8, 64, [128, -5, 40, 7]),        # lengths outside [0, n_kv] are clamped
    (2, 40, 33, 5, 5, 16, [33, 9]),                # widths the tensor cores do not take
    (1, 33, 70, 2, 1, 80, None),
    (1, 9, 20, 3, 3, 256, [19]),
    (1, 7, 6, 3, 1, 8, None),
    (1, 640, 384, 1, 1, 128, None),
    # more query tiles than SMs: whole rounds of pairs, a last round of halves and odd tiles
    (3, 700, 100, 20, 5, 64, [100, 0, 81]),
    (2, 600, 170, 40, 40, 128, [169, 170]),
    (1, 20000, 33, 1, 1, 128, [31]),
    (1, 300, 80, 60, 60, 64, [80]),
]


@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "x".join(map(str, s[:6])))
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_matches_the_definition(shape, dtype):
    c = Case(*shape[:6], lens=shape[6], dtype=dtype)
    c.fwd()
    c.bwd()
    c.check()


@pytest.mark.parametrize("d", [64, 128])
def test_cuda_core_path_matches_too(d):
    c = Case(2, 70, 150, 4, 2, d, lens=[150, 31], path=api.MLA_PATH_SIMT)
    c.fwd()
    c.bwd()
    c.check()


@pytest.mark.parametrize("d", [16, 64, 128])
def test_parts_of_wider_rows(d):
    c = Case(2, 131, 77, 4, 2, d, lens=[77, 50], wide=True)
    assert not c.q.is_contiguous() and not c.k.is_contiguous()
    c.fwd()
    c.bwd()
    c.check()


@pytest.mark.parametrize("d", [32, 64, 128])
def test_masked_states_are_not_used(d):
    """What rows past kv_len hold (NaN, infinities, the largest values) changes no bit."""
    c = Case(2, 140, 300, 4, 2, d, lens=[130, 0])
    c.fwd()
    c.bwd()
    first = [t.clone() for t in (c.out, c.lse, *c.grads)]
    for fill in (float("nan"), float("inf"), -float("inf"), 3e38):
        for t in (c.k, c.v):
            t[0, 130:], t[1] = fill, fill
        c.fwd()
        c.bwd()
        for a, b in zip(first, (c.out, c.lse, *c.grads)):
            assert torch.equal(a, b)
    assert (c.out[1] == 0).all() and torch.isneginf(c.lse[1]).all()
    assert all((t[1] == 0).all() for t in c.grads)
    assert all((t[0, 130:] == 0).all() for t in c.grads[1:])


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("std,scale", [(8.0, 0.25), (1e-3, None), (1.0, 20.0)])
def test_sharp_and_flat_softmax(d, std, scale):
    """Scores of hundreds (the maximum has to move, most exponentials underflow) and of nothing."""
    c = Case(1, 150, 400, 2, 1, d, std=std, scale=scale, seed=3)
    c.fwd()
    c.bwd()
    c.check()


@pytest.mark.parametrize("d", [64, 128])
def test_rising_scores_move_the_maximum_in_every_tile(d):
    """Keys grow along the row, so each tile's maximum passes the last one's by far."""
    c = Case(1, 130, 700, 2, 2, d, seed=4)
    c.q.fill_(0.5)
    ramp = torch.linspace(-4, 4, 700, device="cuda")[None, :, None, None]
    c.k.copy_((ramp + 0.01 * c.k.float()).to(c.dt))
    c.fwd()
    c.bwd()
    c.check()
    c.k.copy_(c.k.flip(1))
    c.fwd()
    c.bwd()
    c.check()


@pytest.mark.parametrize("first", [130, 300])
@pytest.mark.parametrize("n_q", [5, 2500])
@pytest.mark.parametrize("key", [-2.0 ** 66, -float("inf")])
@pytest.mark.parametrize("d,dtype", [(64, "bf16"), (128, "bf16"), (16, "bf16"), (40, "fp32")])
def test_first_states_below_every_score(d, dtype, key, n_q, first):
    """Scores of the first tiles that are -infinity, or overflow to it, weigh nothing; the rest is the
    call on the states behind them, however the states are split over blocks.  (With infinite keys dQ,
    a sum of 0 * infinity, is no number by its definition either.)"""
    c = Case(2, n_q, 400, 4, 2, d, lens=[400, 350], dtype=dtype, scale=0.25, seed=8)
    c.q[..., 0] = 2.0 ** 64
    c.k[..., 0] *= 2.0 ** -64
    c.k[:, :first, :, 0] = key                     # 2^64 2^66 / 4 is 2^128
    c.fwd()
    if np.isfinite(key):
        c.bwd()
    part = object.__new__(Case)
    part.__dict__.update(c.__dict__)
    part.cc = api.make_cross_config(batch=2, n_heads=4, n_kv_heads=2, d_head=d, n_q=n_q,
                                    n_kv=400 - first, softmax_scale=0.25, dtype=dtype)
    part.lens = [400 - first, 350 - first]
    part.k, part.v = c.k[:, first:], c.v[:, first:]
    part.grads = [c.grads[0], *(t[:, first:] for t in c.grads[1:])]
    part.check(backward=np.isfinite(key))
    if np.isfinite(key):
        assert all((t[:, :first] == 0).all() for t in c.grads[1:])


@pytest.mark.parametrize("d,dtype", [(64, "bf16"), (128, "bf16"), (40, "fp32")])
def test_the_smallest_scales_weigh_every_state_alike(d, dtype):
    for n_q in (3, 300):
        c = Case(2, n_q, 100, 2, 1, d, lens=[100, 41], dtype=dtype, scale=1e-42)
        c.q[:, ::2] = 0
        c.fwd()
        c.bwd()
        c.check()


@pytest.mark.parametrize("d", [16, 64, 128])
def test_same_call_same_bits_and_no_writes_outside(d):
    c = Case(2, 150, 260, 6, 2, d, lens=[260, 101])
    c.fwd()
    c.bwd()
    first = [t.clone() for t in (c.out, c.lse, *c.grads)]
    c.ws.fill_(0)
    for _ in range(3):
        c.fwd()
        c.bwd()
    for a, b in zip(first, (c.out, c.lse, *c.grads)):
        assert torch.equal(a, b)
    # the same outputs inside larger buffers: what lies around them stays
    whole = []
    for t in (c.out, c.lse, *c.grads):
        pad = torch.full((t.numel() + 2048,), 5.0, device="cuda", dtype=t.dtype)
        whole.append((pad, pad[1024:1024 + t.numel()].view(t.shape)))
    c.out, c.lse, *c.grads = [v for _, v in whole]
    c.fwd()
    c.bwd()
    for a, (pad, v) in zip(first, whole):
        assert torch.equal(a, v)
        assert (pad[:1024] == 5).all() and (pad[1024 + a.numel():] == 5).all()


def test_lse_is_optional():
    c = Case(1, 20, 90, 2, 2, 128)
    c.fwd()
    out = c.out.clone()
    c.out.zero_()
    c.fwd(lse=False)
    assert torch.equal(out, c.out)


@pytest.mark.parametrize("d", [64, 128])
def test_other_stream_and_graph(d):
    """Two captured calls that share a workspace, replayed in turn on a side stream, while eager
    calls of the same arrays run before and after."""
    c = Case(2, 140, 200, 4, 2, d, lens=[200, 90])
    e = Case(1, 70, 512, 4, 4, d, seed=9)
    need = max(c.ws.numel(), e.ws.numel())
    c.ws = e.ws = torch.zeros(need, device="cuda", dtype=torch.uint8)
    want = []
    for x in (c, e):
        x.fwd()
        x.bwd()
        want.append([t.clone() for t in (x.out, x.lse, *x.grads)])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graphs = []
    for x in (c, e):
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr, stream=side, capture_error_mode="relaxed"):
            x.fwd()
            x.bwd()
        graphs.append(gr)
    for x in (c, e):
        for t in (x.out, x.lse, *x.grads):
            t.zero_()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for _ in range(2):
            for gr in graphs:
                gr.replay()
    side.synchronize()
    for x, w in zip((c, e), want):
        for a, b in zip(w, (x.out, x.lse, *x.grads)):
            assert torch.equal(a, b)
    c.fwd(stream=side)
    c.bwd(stream=side)
    side.synchronize()
    c.check()


def test_gradient_against_differences():
    """fp32: f = sum(g out) at q +- h u: the difference quotient is off by O(h^2) f''' and by the
    outputs' fp32 error / h; with h = 1e-2 and |u| = 1 both stay below 2e-3 of the gradient's
    scale sqrt(sum grad^2)."""
    c = Case(1, 6, 30, 2, 1, 64, dtype="fp32", seed=5)
    c.fwd()
    c.bwd()
    f = lambda: float((c.g.double() * c.out.double()).sum())
    for t, grad in zip((c.q, c.k, c.v), c.grads):
        u = torch.randn(t.shape, device="cuda", generator=torch.Generator("cuda").manual_seed(6))
        u /= u.norm()
        old, h, at = t.clone(), 1e-2, []
        for s in (h, -h):
            t.copy_(old + s * u)
            c.fwd()
            at.append(f())
        t.copy_(old)
        assert abs((at[0] - at[1]) / (2 * h) - float((grad * u).sum())) < 2e-3 * float(grad.norm())


def test_encoder_states_serve_chunks_and_training():
    """A prompt attended by calls of several lengths, and its gradients."""
    c = Case(2, 60, 77, 4, 2, 128, lens=[77, 20])
    e = rollout.EncoderStates(c.k, c.v, n_heads=4, kv_len=c.kv_len)
    e.attend(c.q, c.out, lse=c.lse)
    e.backward(c.q, c.out, c.lse, c.g, *c.grads)
    c.check()
    one = torch.empty_like(c.out[:, :1])
    q1 = c.q[:, 7:8].contiguous()
    e.attend(q1, one)
    lens = [77, 20]
    np64 = lambda t: t.double().cpu().numpy()
    out, _, e_out, _ = oracle.cross_attention(np64(q1), np64(c.k), np64(c.v), lens,
                                              c.cc.softmax_scale, p_rel=P_REL)
    close("one", np64(one), out, e_out * (1 + BF16) + BF16 * np.abs(out))
    assert int(e.dev_status) == 0


def test_encoder_states_on_a_side_stream():
    """The workspace that a backward call makes is memory of the stream it runs on: a block just freed
    on the current stream, behind work that has yet to read and write it, is not taken."""
    c = Case(2, 60, 300, 4, 2, 128, lens=[300, 20])
    e = rollout.EncoderStates(c.k, c.v, n_heads=4, kv_len=c.kv_len)
    side = torch.cuda.Stream()
    block = torch.full_like(c.ws, 5)
    torch.cuda.synchronize()
    torch.cuda._sleep(100_000_000)                          # some 50 ms on the current stream
    kept = block.clone()
    block.fill_(0x7F)
    del block
    e.attend(c.q, c.out, lse=c.lse, stream=side)
    e.backward(c.q, c.out, c.lse, c.g, *c.grads, stream=side)
    torch.cuda.synchronize()
    c.check()
    assert (kept == 5).all() and int(e.dev_status) == 0


def test_layer_sized_call():
    """A chunk of the Wan-shaped layer against prompts of two lengths: every element of the first and
    the last head (whose keys no other head shares) against the definition."""
    lens = [512, 389]
    c = Case(2, 4680, 512, 12, 12, 128, lens=lens, seed=11)
    c.fwd()
    c.bwd()
    for h in (0, 11):
        part = object.__new__(Case)
        one = lambda t: t[:, :, h:h + 1]
        part.cc = api.make_cross_config(batch=2, n_heads=1, n_kv_heads=1, d_head=128, n_q=4680,
                                        n_kv=512)
        part.dt, part.lens, part.status = c.dt, lens, c.status
        part.q, part.k, part.v, part.g, part.out = map(one, (c.q, c.k, c.v, c.g, c.out))
        part.lse = c.lse[:, h:h + 1]
        part.grads = [one(t) for t in c.grads]
        part.check()


def test_gradients_of_many_queries_per_state_tile():
    """Several blocks share a tile's queries and their sums are added; one block writes its own."""
    for B, n_q, n_kv, H, Hkv, d, lens in ((1, 900, 100, 4, 1, 64, [99]), (1, 1500, 300, 2, 2, 128, [130]),
                                          (2, 81, 129, 2, 1, 128, [129, 0])):
        c = Case(B, n_q, n_kv, H, Hkv, d, lens=lens, seed=12)
        c.fwd()
        c.bwd()
        c.check()
        first = [t.clone() for t in c.grads]
        for _ in range(3):
            c.bwd()
        assert all(torch.equal(a, b) for a, b in zip(first, c.grads))


def test_calls_on_two_streams_at_once():
    """Forward and backward of two problems side by side, each with its own workspace."""
    a, b = Case(2, 700, 300, 4, 2, 128, lens=[300, 41]), Case(3, 500, 200, 8, 8, 64, seed=5)
    want = []
    for c in (a, b):
        c.fwd()
        c.bwd()
        want.append([t.clone() for t in (c.out, c.lse, *c.grads)])
        for t in (c.out, c.lse, *c.grads):
            t.zero_()
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(5):
        for c, s in zip((a, b), streams):
            c.fwd(stream=s)
            c.bwd(stream=s)
    torch.cuda.synchronize()
    for c, w in zip((a, b), want):
        assert all(torch.equal(x, y) for x, y in zip(w, (c.out, c.lse, *c.grads)))
        assert int(c.status) == 0


@pytest.mark.parametrize("shape", [
    (1, 700, 300, 4, 4, 128, [300]),               # blocks share a tile of states: sums in dQ
    (3, 260, 333, 8, 2, 64, [333, 0, 130]),
    (4, 90, 300, 40, 40, 128, [300, 1, 0, 200]),   # a block per tile
    (2, 40, 129, 3, 1, 64, [0, 0]),                # nothing to attend to
], ids=lambda s: "x".join(map(str, s[:6])))
def test_calls_behind_one_another_see_each_other(shape):
    """Every launch of a chain of forward and backward calls may start before the one in front of it
    has ended.  With one workspace, outputs written over and inputs changed between the calls, the
    chain has to give the bits of calls that run one at a time; the chain is run eagerly and as a
    graph."""
    B, n_q, n_kv, H, Hkv, d, lens = shape
    c = Case(B, n_q, n_kv, H, Hkv, d, lens=lens, seed=12)
    steps = 6
    inputs = [c.q.clone(), c.k.clone(), c.v.clone(), c.g.clone()]
    results = [[torch.empty_like(t) for t in (c.out, *c.grads)] for _ in range(steps)]

    def restore():
        for t, u in zip((c.q, c.k, c.v, c.g), inputs):
            t.copy_(u)
        c.ws.fill_(0xFF)

    def chain(wait):
        for step in range(steps):
            c.fwd()
            wait()
            c.bwd()
            wait()
            for to, t in zip(results[step], (c.out, *c.grads)):
                to.copy_(t)
            # The next inputs are this call's results: a late write or an early read would show.  (Only
            # a part of them, or the scores grow with every step, in float64 too: to 1e10 in six, where
            # an fp32 lse is off by 2^-24 1e10 = 600 and exp(x - lse) may be anything.)
            c.q.copy_(c.grads[0] / 64 + inputs[0])
            c.k.copy_(c.grads[1] / 64 + inputs[1])
            c.v.copy_(c.grads[2] / 64 + inputs[2])
            c.g.copy_(c.out / 64 + inputs[3])
            wait()

    restore()
    chain(torch.cuda.synchronize)
    want = [[t.clone() for t in r] for r in results]
    assert all(torch.isfinite(t).all() for r in want for t in r)

    def check():
        torch.cuda.synchronize()
        assert int(c.status) == 0
        for got, ref in zip(results, want):
            assert all(torch.equal(a, b) for a, b in zip(got, ref))
            for t in got:
                t.fill_(7.0)

    for _ in range(5):
        restore()
        chain(lambda: None)
        check()
    restore()
    graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(graph, stream=side):
        chain(lambda: None)
    for _ in range(5):
        restore()
        graph.replay()
        check()


@pytest.mark.parametrize("d", [64, 128])
def test_lengths_and_inputs_rewritten_between_calls(d):
    """Small calls in one chain, eager and as a graph, with the lengths, the inputs and the workspace's
    statistics rewritten between them: each call sees what was written just before it."""
    c = Case(3, 40, 200, 2, 2, d, lens=[200, 200, 200], seed=13)
    steps = 12
    g = torch.Generator(device="cuda").manual_seed(14)
    lens = torch.randint(0, 201, (steps, 3), generator=g, device="cuda", dtype=torch.int32)
    qs = torch.randn((steps, *c.q.shape), generator=g, device="cuda").to(c.dt)
    results = [[torch.empty_like(t) for t in (c.out, c.lse, *c.grads)] for _ in range(steps)]

    def chain(wait):
        for step in range(steps):
            c.kv_len.copy_(lens[step])
            c.q.copy_(qs[step])
            wait()
            c.fwd()
            wait()
            c.bwd()
            wait()
            for to, t in zip(results[step], (c.out, c.lse, *c.grads)):
                to.copy_(t)

    chain(torch.cuda.synchronize)
    want = [[t.clone() for t in r] for r in results]

    def check():
        torch.cuda.synchronize()
        assert int(c.status) == 0
        for got, ref in zip(results, want):
            assert all(torch.equal(a, b) for a, b in zip(got, ref))
            for t in got:
                t.fill_(7.0)

    check()
    for _ in range(10):
        chain(lambda: None)
        check()
    graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(graph, stream=side):
        chain(lambda: None)
    for _ in range(10):
        graph.replay()
        check()


@pytest.mark.parametrize("d", [64, 128])
def test_arrays_of_almost_2_to_31_elements(d):
    """Rows whose byte offsets (and, for 64-bit reads of the arrays, element offsets) are near the
    largest allowed.  Only the first and the last 64 queries have an upstream gradient, so dK and dV
    are those of a call with these 128 queries alone; the others' dQ is exactly zero."""
    H, n_kv, ends = 12, 70, 64
    n_q = (2 ** 31 - 1) // (H * d) - 1
    n_q -= n_q % 80 - 17                       # a ragged last tile
    small = Case(1, 2 * ends, n_kv, H, 3, d, seed=3)
    small.fwd()
    small.bwd()
    small.check()
    c = Case(1, 1, n_kv, H, 3, d)              # (a config and buffers to widen)
    cc = api.make_cross_config(batch=1, n_heads=H, n_kv_heads=3, d_head=d, n_q=n_q, n_kv=n_kv)
    new = lambda: torch.zeros((1, n_q, H, d), device="cuda", dtype=torch.bfloat16)
    q, g, out, d_q = new(), new(), new(), new().fill_(7.0)
    lse = torch.zeros((1, H, n_q), device="cuda")
    pick = lambda t: torch.cat((t[:, :ends], t[:, -ends:]), 1)
    for big, part in ((q, small.q), (g, small.g)):
        big[:, :ends], big[:, -ends:] = part[:, :ends], part[:, ends:]
    api.mla_cross_attention_fwd(cc, q, small.k, small.v, out, lse=lse, dev_status=c.status)
    ws = torch.empty(api.mla_cross_attention_bwd_workspace_bytes(cc), device="cuda",
                     dtype=torch.uint8)
    d_k, d_v = torch.empty_like(small.k), torch.empty_like(small.v)
    api.mla_cross_attention_bwd(cc, q, small.k, small.v, out, lse, g, d_q, d_k, d_v, ws,
                                dev_status=c.status)
    assert int(c.status) == 0
    # a row's results take no part of other rows (one tile of states or one rescaling rule a warp
    # apart: within two roundings to bf16)
    for got, want in ((pick(out), small.out), (pick(d_q), small.grads[0])):
        err = (got.float() - want.float()).abs()
        assert (err <= 2 * BF16 * want.float().abs() + 1e-5).all()
    assert (pick(lse.transpose(1, 2)) - small.lse.transpose(1, 2)).abs().max() <= 2.0 ** -20
    assert (d_q[:, ends:-ends] == 0).all()
    # the same 128 terms in fp32, summed in another order: 128 roundings of 2^-24 of the terms' sum of
    # magnitudes, below 2^-10 here, and one rounding to bf16 each
    for got, want in ((d_k, small.grads[1]), (d_v, small.grads[2])):
        err = (got.float() - want.float()).abs()
        assert (err <= 2 * BF16 * want.float().abs() + 2.0 ** -10).all()


def test_bad_pointers_are_refused():
    c = Case(1, 8, 16, 2, 2, 64)
    host = torch.zeros(c.q.shape, dtype=c.dt)
    with pytest.raises(api.MLAError):
        api.mla_cross_attention_fwd(c.cc, host, c.k, c.v, c.out)
    flat = torch.zeros(c.q.numel() + 8, device="cuda", dtype=c.dt)
    off = flat[1:1 + c.q.numel()].view(c.q.shape)
    with pytest.raises(api.MLAError):
        api.mla_cross_attention_fwd(c.cc, off, c.k, c.v, c.out)
    c.fwd()
    with pytest.raises(api.MLAError):
        api.mla_cross_attention_bwd(c.cc, c.q, c.k, c.v, c.out, c.lse, c.g, *c.grads, c.ws[:128])
    with pytest.raises(api.MLAError):
        api.mla_cross_attention_bwd(c.cc, c.q, c.k, c.v, c.out, None, c.g, *c.grads, c.ws)
