"""GPU parity of the long-history operators against oracle/long_history.py (fp64).

Tolerances, stated per element from the rounding points (half a bf16 step is 2^-8 of the value):
* attention: the weights P enter the value product as bf16, which spreads to 2^-8 P|V|; the result
  is rounded once, 2^-8 |ref|; the fp32 scores, exponentials and sums take 2^-11 P|V| (a score of
  128 products of magnitude up to a few tens carries at most about 128 2^-24 60 = 2^-11);
* lse: 2^-11 on the scores as above, in fp32;
* gradients: dS and P enter their products as bf16 (2^-8 |dS|), the forward's bf16 output enters
  rowsum(dO * O) (2^-8 P |dO||O|), the result is rounded once, and the fp32 part takes 2^-11 of the
  absolute terms before cancellation;
* rotation: one rounding to the type, 2^-22 of the two terms for the fp32 sine, cosine and products
  (each within 2^-23), summed over both.
"""

import numpy as np
import pytest
import torch

import oracle
import oracle.long_history as lh
from candidate_isolated_jagged_b200 import jca
from helpers import dev

pytestmark = pytest.mark.gpu

HALF = {torch.bfloat16: 2.0**-8, torch.float16: 2.0**-11, torch.float32: 2.0**-24}
EDGES = [1, 5, 0, 17, 64, 127, 128, 129, 255, 256, 257, 300, 513, 2]


def near(got, ref, tol, what):
    got = got.double().cpu().numpy()
    assert got.shape == ref.shape
    assert np.all(np.isfinite(got)), f"{what}: not finite"
    over = np.abs(got - ref) - tol
    at = np.unravel_index(np.argmax(over), over.shape) if over.size else ()
    assert over.size == 0 or over[at] <= 0, f"{what}: {got[at]} against {ref[at]} +- {tol[at]} at {at}"


class Window:
    """A batch for the windowed attention, on the GPU, and the oracle's view of it."""

    def __init__(self, lengths, H, Hkv, d, seed=0, valid=None, idx=torch.int64, fused=False, junk=None):
        g = torch.Generator().manual_seed(seed)
        self.off_np = np.concatenate([[0], np.cumsum(lengths)]).astype(np.int64)
        T = self.T = int(self.off_np[-1])
        x = torch.randn(T, H + 2 * Hkv, d, generator=g).to(torch.bfloat16)
        self.do = torch.randn(T, H, d, generator=g).to(torch.bfloat16)
        self.valid_np = None if valid is None else np.asarray(valid, dtype=np.uint8)
        self.valid = None
        if valid is not None:
            self.valid = torch.tensor(self.valid_np, device=dev())
            if junk is not None:
                x[self.valid_np == 0] = junk
                self.do[self.valid_np == 0] = junk
        self.H, self.Hkv, self.d, self.scale = H, Hkv, d, 1.0 / np.sqrt(d)
        self.q_cpu, self.k_cpu, self.v_cpu = x.split([H, Hkv, Hkv], 1)
        on = x.to(dev()).split([H, Hkv, Hkv], 1)
        self.q, self.k, self.v = on if fused else [t.contiguous() for t in on]
        self.dout = self.do.to(dev())
        self.off = torch.tensor(self.off_np, dtype=idx, device=dev())
        self.st = jca.new_status(dev())

    def forward(self, window, sinks, lse=True, **kw):
        self.out = torch.full((self.T, self.H, self.d), float("nan"), dtype=torch.bfloat16, device=dev())
        self.lse = torch.full((self.T, self.H), float("nan"), device=dev()) if lse else None
        jca.jagged_window_attn_fwd(self.q, self.k, self.v, self.out, self.off, window, sinks,
                                   valid=self.valid, lse=self.lse, status=self.st, **kw)
        return self.out

    def users(self, window, sinks):
        for s, e in zip(self.off_np[:-1], self.off_np[1:]):
            if e > s:
                va = None if self.valid_np is None else self.valid_np[s:e]
                yield slice(int(s), int(e)), lh.window_mask(int(e - s), window, sinks, va)

    def check_forward(self, window, sinks, what=""):
        torch.cuda.synchronize()
        jca.check_status(self.st, what)
        for r, mask in self.users(window, sinks):
            ref, lse, _, A = lh.masked(self.q_cpu[r], self.k_cpu[r], self.v_cpu[r], mask, self.scale)
            near(self.out[r], ref, (2.0**-8 + 2.0**-11) * A + 2.0**-8 * np.abs(ref) + 1e-30, what)
            if self.lse is not None:
                live = mask.any(1)
                got = self.lse[r].double().cpu().numpy()
                assert np.all(got[~live] == -np.inf), what
                assert np.max(np.abs(got[live] - lse[live]), initial=0.0) <= 2.0**-11, what

    def backward(self, window, sinks, **kw):
        """The gradients for the oracle's output and log-sum-exp, rounded to the stored types."""
        out = np.zeros((self.T, self.H, self.d))
        lse = np.full((self.T, self.H), -np.inf)
        for r, mask in self.users(window, sinks):
            out[r], lse[r], _, _ = lh.masked(self.q_cpu[r], self.k_cpu[r], self.v_cpu[r], mask, self.scale)
        self.out = torch.tensor(out).to(torch.bfloat16).to(dev())
        self.lse = torch.tensor(lse).float().to(dev())
        if self.valid_np is not None:
            self.out[self.valid == 0] = float("nan")
            self.lse[self.valid == 0] = float("nan")
        n = dict(dtype=torch.bfloat16, device=dev())
        self.grads = [torch.full((self.T, h, self.d), float("nan"), **n) for h in (self.H, self.Hkv, self.Hkv)]
        jca.jagged_window_attn_bwd(self.q, self.k, self.v, self.out, self.dout, self.lse, *self.grads,
                                   self.off, window, sinks, valid=self.valid, status=self.st, **kw)
        return self.grads

    def check_backward(self, window, sinks, what=""):
        torch.cuda.synchronize()
        jca.check_status(self.st, what)
        for r, mask in self.users(window, sinks):
            ref, tol = lh.gradients(self.q_cpu[r], self.k_cpu[r], self.v_cpu[r], self.do[r], mask, self.scale)
            for name, got, x, (soft, hard) in zip(("dq", "dk", "dv"), self.grads, ref, tol):
                near(got[r], x, 2.0**-8 * soft + 2.0**-11 * hard + 2.0**-8 * np.abs(x) + 1e-30,
                     f"{what} {name}")


# ------------------------------------------------------------------------------------------------
# Windowed attention
# ------------------------------------------------------------------------------------------------

WINDOWS = [(1, 0), (1, 3), (2, 1), (40, 0), (100, 4), (128, 128), (129, 16), (1 << 40, 0), (300, 1)]


@pytest.mark.parametrize("d", [16, 32, 64, 128])
@pytest.mark.parametrize("window,sinks", WINDOWS)
def test_window_forward_edges(d, window, sinks):
    b = Window(EDGES, 2, 2, d, seed=d)
    b.forward(window, sinks)
    b.check_forward(window, sinks, f"d={d} w={window} s={sinks}")


@pytest.mark.parametrize("d", [16, 32, 64, 128])
@pytest.mark.parametrize("window,sinks", WINDOWS)
def test_window_backward_edges(d, window, sinks):
    b = Window(EDGES, 2, 2, d, seed=d + 1)
    b.backward(window, sinks)
    b.check_backward(window, sinks, f"d={d} w={window} s={sinks}")


@pytest.mark.parametrize("lengths", [[1], [1] * 300, [3, 2] * 90, [700], [0, 0, 5, 0], [2000]])
@pytest.mark.parametrize("H,Hkv", [(4, 1), (6, 2)])
def test_window_shapes(lengths, H, Hkv):
    b = Window(lengths, H, Hkv, 32, seed=len(lengths), idx=torch.int32)
    b.forward(70, 2)
    b.check_forward(70, 2)
    b.backward(70, 2)
    b.check_backward(70, 2)


@pytest.mark.parametrize("fill", [float("nan"), float("inf"), -3e38])
@pytest.mark.parametrize("d", [16, 64, 128])
def test_window_padding_holds_anything(d, fill):
    """Padding in front, in holes, at the end, a user of padding alone; its q, k, v, dO, O and lse are
    not finite."""
    lengths = [40, 200, 16, 513, 130]
    rng = np.random.default_rng(5)
    valid = (rng.random(sum(lengths)) > 0.3).astype(np.uint8)
    valid[:9] = 0
    valid[240:256] = 0
    valid[-70:] = 0
    b = Window(lengths, 4, 2, d, seed=2, valid=valid, junk=fill)
    out = b.forward(90, 5)
    b.check_forward(90, 5)
    assert bool((out[b.valid == 0] == 0).all())
    grads = b.backward(90, 5)
    b.check_backward(90, 5)
    for g in grads:
        assert bool((g[b.valid == 0] == 0).all())


def test_window_fused_projection_rows():
    b = Window([100, 31, 260], 4, 2, 64, seed=3, fused=True)
    assert not b.q.is_contiguous()
    b.forward(50, 3)
    b.check_forward(50, 3)
    b.backward(50, 3)
    b.check_backward(50, 3)


def test_window_as_long_as_the_row_is_the_causal_layer():
    b = Window([300, 7, 129, 650], 4, 4, 128, seed=4)
    got = b.forward(650, 0, lse=False)
    ref = torch.empty_like(got)
    st = jca.new_status(dev())
    jca.jagged_causal_attn_fwd(b.q, b.k, b.v, ref, b.off, status=st)
    jca.check_status(st)
    torch.testing.assert_close(got.float(), ref.float(), atol=3e-2, rtol=2.0**-6)


def test_window_scale_and_equal_bits():
    b = Window([90, 400], 2, 1, 64, seed=6)
    b.scale = 0.05
    b.forward(64, 2, scale=0.05)
    b.check_forward(64, 2)
    g1 = [g.clone() for g in b.backward(64, 2, scale=0.05)]
    b.check_backward(64, 2)
    for _ in range(3):
        for x, y in zip(g1, b.backward(64, 2, scale=0.05)):
            assert torch.equal(x, y)


def test_window_large_scores():
    """Scores of some hundreds: the running maximum moves by more than any rescaling threshold."""
    b = Window([400, 30], 2, 2, 64, seed=7)
    ramp = torch.linspace(0.05, 6.0, b.T)[:, None, None]
    b.k_cpu = (b.k_cpu.float() * ramp).to(torch.bfloat16)
    b.k = b.k_cpu.to(dev())
    b.forward(1000, 0, lse=False)
    torch.cuda.synchronize()
    # a score of 64 products of magnitude up to 6 * 4 * 4 carries up to 64 2^-24 100 = 2^-11 as well
    b.check_forward(1000, 0)
    b.backward(1000, 0)
    b.check_backward(1000, 0)


def test_window_empty_batches():
    for lengths in ([], [0], [0, 0, 0]):
        b = Window(lengths, 2, 2, 16)
        b.forward(4, 1)
        b.backward(4, 1)
        torch.cuda.synchronize()
        jca.check_status(b.st)


@pytest.mark.parametrize("off", [[0, 10, 9], [1, 5, 13], [0, 5, 12], [0, -3, 13], [0, 5, 1 << 40]])
def test_window_bad_offsets_write_nothing(off):
    b = Window([4, 9], 2, 2, 16)
    b.off = torch.tensor(off, device=dev())
    out = torch.full((13, 2, 16), 7.0, dtype=torch.bfloat16, device=dev())
    lse = torch.full((13, 2), 7.0, device=dev())
    grads = [torch.full_like(out, 7.0) for _ in range(3)]
    jca.jagged_window_attn_fwd(b.q, b.k, b.v, out, b.off, 4, 1, lse=lse, status=b.st)
    torch.cuda.synchronize()
    assert int(b.st.item()) == 2
    st = jca.new_status(dev())
    jca.jagged_window_attn_bwd(b.q, b.k, b.v, out, out, lse, *grads, b.off, 4, 1, status=st)
    torch.cuda.synchronize()
    assert int(st.item()) == 2
    for x in [out, lse] + grads:
        assert bool((x == 7.0).all())


def test_window_captured_and_replayed_with_an_eager_call_between():
    """One graph of forward and backward, replayed on new inputs; an eager call of another batch
    with its own workspace runs between the replays."""
    b = Window([200, 33, 300], 4, 2, 64, seed=8)
    other = Window([77, 500], 4, 2, 64, seed=9)
    ws = torch.empty(jca.jca_window_workspace_bytes(3, b.T, 4, 2, 64, 2), dtype=torch.uint8, device=dev())
    wb = torch.empty(jca.jca_window_bwd_workspace_bytes(3, b.T, 4, 2, 64, 2), dtype=torch.uint8, device=dev())
    out, lse = torch.empty_like(b.q), torch.empty(b.T, 4, device=dev())
    grads = [torch.empty_like(x) for x in (b.q, b.k, b.v)]

    def step():
        jca.jagged_window_attn_fwd(b.q, b.k, b.v, out, b.off, 60, 2, lse=lse, workspace=ws, status=b.st)
        jca.jagged_window_attn_bwd(b.q, b.k, b.v, out, b.dout, lse, *grads, b.off, 60, 2, workspace=wb,
                                   status=b.st)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for seed in (1, 2):
        g = torch.Generator().manual_seed(seed)
        for x in (b.q, b.k, b.v, b.dout):
            x.copy_(torch.randn(x.shape, generator=g).to(torch.bfloat16))
        other.forward(60, 2)
        graph.replay()
        torch.cuda.synchronize()
        kept = [x.clone() for x in [out, lse] + grads]
        step()
        torch.cuda.synchronize()
        for x, y in zip(kept, [out, lse] + grads):
            assert torch.equal(x, y)
    other.check_forward(60, 2)


def test_window_numbers_past_the_c_types():
    b = Window([70, 40], 2, 2, 16, seed=16)
    b.forward(1 << 70, 0)
    b.check_forward(1 << 40, 0)
    with pytest.raises(jca.JcaError):
        b.forward(20, (1 << 32) + 1)
    d = Decode([5], [8], 2, 2, 16, seed=16)
    d.run(1 << 70, 1 << 70)
    d.check(1 << 40, 1 << 40)
    t = Tree([3], [9], 2, 2, 16, seed=16)
    with pytest.raises(jca.JcaError):
        t.run((1 << 32) + 3)


def test_window_two_streams():
    batches = [Window([150, 420, 64], 4, 4, 64, seed=s) for s in (11, 12)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in batches]
    for _ in range(3):
        for b, s in zip(batches, streams):
            with torch.cuda.stream(s):
                b.forward(100, 4)
    torch.cuda.synchronize()
    for b in batches:
        b.check_forward(100, 4)


def test_calls_on_a_given_stream_make_their_scratch_there():
    """With a stream and no workspace or status, the scratch must outlive the call: memory of its
    size is taken and overwritten on the current stream while the given stream is still busy."""
    b, t = Window([150, 420, 64], 4, 4, 64, seed=13), Tree([9, 20], [200, 77], 4, 2, 64, seed=13)
    side, busy = torch.cuda.Stream(), torch.randn(4096, 4096, device=dev())
    b.forward(100, 4)
    b.backward(100, 4)
    want = [b.out.clone()] + [x.clone() for x in b.grads]
    got = [torch.full_like(x, float("nan")) for x in want]
    lse = b.lse
    fwd = torch.empty_like(lse)
    n = [jca.jca_window_workspace_bytes(3, b.T, 4, 4, 64, 4),
         jca.jca_window_bwd_workspace_bytes(3, b.T, 4, 4, 64, 4), 4]
    fresh = torch.empty_like(b.out)
    for handle in (side, side.cuda_stream):
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            for _ in range(20):
                busy = busy @ busy * 1e-2
        jca.jagged_window_attn_fwd(b.q, b.k, b.v, fresh, b.off, 100, 4, lse=fwd, stream=handle)
        jca.jagged_window_attn_bwd(b.q, b.k, b.v, b.out, b.dout, lse, *got[1:], b.off, 100, 4, stream=handle)
        jca.cand_tree_attn_fwd(t.q, t.k, t.v, t.off, t.parent, t.hk, t.hv, t.ho, t.out, 20, stream=handle)
        junk = [torch.full((x,), 255, dtype=torch.uint8, device=dev()) for x in n for _ in range(4)]
        torch.cuda.synchronize()
        del junk
        for x, y in zip(got[1:], want[1:]):
            assert torch.equal(x, y)
        t.check()
        b.out, b.lse = fresh, fwd
        b.check_forward(100, 4)
        b.out, b.lse = want[0], lse
        for x in got + [fresh, fwd, t.out]:
            x.fill_(float("nan"))


def test_window_writes_its_rows_only():
    """Gradients and outputs that lie inside larger buffers: the rows before and behind stay. The
    last user is shorter than the first tokens of the call."""
    b = Window([300, 140, 3], 4, 2, 32, seed=14)
    big = {n: torch.full((b.T + 64, h, 32), 3.0, dtype=torch.bfloat16, device=dev())
           for n, h in (("out", 4), ("dq", 4), ("dk", 2), ("dv", 2))}
    lse = torch.full((b.T + 64, 4), 3.0, device=dev())
    mid = slice(32, 32 + b.T)
    for window, sinks in ((2, 8), (1, 128), (50, 5)):
        b.backward(window, sinks)
        want = b.grads
        jca.jagged_window_attn_fwd(b.q, b.k, b.v, big["out"][mid], b.off, window, sinks, lse=lse[mid], status=b.st)
        jca.jagged_window_attn_bwd(b.q, b.k, b.v, b.out, b.dout, b.lse, *(big[n][mid] for n in ("dq", "dk", "dv")),
                                   b.off, window, sinks, status=b.st)
        for n, w in zip(("dq", "dk", "dv"), want):
            assert torch.equal(big[n][mid], w)
        b.check_backward(window, sinks)
        b.out, b.lse = big["out"][mid], lse[mid]
        b.check_forward(window, sinks)
        for x in list(big.values()) + [lse]:
            assert bool((x[:32] == 3.0).all()) and bool((x[32 + b.T:] == 3.0).all())


def test_window_backward_on_many_users_twice():
    """More users than units run at once, and equal bits from equal calls."""
    rng = np.random.default_rng(3)
    b = Window(list(rng.integers(0, 120, 700)), 2, 1, 64, seed=15)
    first = [x.clone() for x in b.backward(20, 3)]
    again = b.backward(20, 3)
    for x, y in zip(first, again):
        assert torch.equal(x, y)
    b.check_backward(20, 3)


def test_window_rows_beyond_32_bit_offsets():
    """2^31 elements and more in q and out; sampled users at both ends."""
    lengths = [1000] * 1050
    H, d = 16, 128
    T = sum(lengths)
    assert T * H * d > 2**31
    off = torch.arange(1051, device=dev()) * 1000
    g = torch.Generator(device=dev()).manual_seed(0)
    q = torch.empty(T, H, d, dtype=torch.bfloat16, device=dev()).normal_(generator=g)
    k, v = (torch.empty(T, 1, d, dtype=torch.bfloat16, device=dev()).normal_(generator=g) for _ in range(2))
    out, lse, st = torch.empty_like(q), torch.empty(T, H, device=dev()), jca.new_status(dev())
    jca.jagged_window_attn_fwd(q, k, v, out, off, 64, 4, lse=lse, status=st)
    jca.check_status(st)
    mask, ends = lh.window_mask(1000, 64, 4), [slice(0, 1000), slice(T - 1000, T)]
    for r in ends:
        ref, _, _, A = lh.masked(q[r], k[r], v[r], mask, d**-0.5)
        near(out[r], ref, (2.0**-8 + 2.0**-11) * A + 2.0**-8 * np.abs(ref), f"rows {r}")
        out[r] = torch.tensor(ref).to(torch.bfloat16)
    dq, dk, dv = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)
    jca.jagged_window_attn_bwd(q, k, v, out, q, lse, dq, dk, dv, off, 64, 4, status=st)
    jca.check_status(st)
    for r in ends:
        ref, tol = lh.gradients(q[r], k[r], v[r], q[r], mask, d**-0.5)
        for name, got, x, (soft, hard) in zip(("dq", "dk", "dv"), (dq, dk, dv), ref, tol):
            near(got[r], x, 2.0**-8 * soft + 2.0**-11 * hard + 2.0**-8 * np.abs(x), f"rows {r} {name}")


# ------------------------------------------------------------------------------------------------
# One token over a cache
# ------------------------------------------------------------------------------------------------

class Decode:
    def __init__(self, lens, caps, H, Hkv, d, seed=0, idx=torch.int64, junk=float("nan"), spare=3):
        g = torch.Generator().manual_seed(seed)
        self.lens, B = list(lens), len(lens)
        self.off_np = np.concatenate([[0], np.cumsum(caps)]).astype(np.int64)
        R = int(self.off_np[-1]) + spare
        self.q_cpu, self.kn_cpu, self.vn_cpu = (torch.randn(B, h, d, generator=g).to(torch.bfloat16)
                                                for h in (H, Hkv, Hkv))
        self.kc_cpu, self.vc_cpu = (torch.randn(R, Hkv, d, generator=g).to(torch.bfloat16) for _ in range(2))
        used = np.zeros(R, bool)
        for b, n in enumerate(self.lens):
            used[self.off_np[b]:self.off_np[b] + max(n, 0)] = True
        self.kc_cpu[~used] = junk
        self.vc_cpu[~used] = junk
        to = lambda x: x.to(dev())                                  # noqa: E731
        self.q, self.kn, self.vn = to(self.q_cpu), to(self.kn_cpu), to(self.vn_cpu)
        self.kc, self.vc = to(self.kc_cpu), to(self.vc_cpu)
        self.off = torch.tensor(self.off_np, dtype=idx, device=dev())
        self.len = torch.tensor(self.lens, dtype=idx, device=dev())
        self.out = torch.full((B, H, d), float("nan"), dtype=torch.bfloat16, device=dev())
        self.scale, self.st = d**-0.5, jca.new_status(dev())

    def run(self, window, sinks):
        jca.jagged_window_decode_fwd(self.q, self.kn, self.vn, self.kc, self.vc, self.out, self.off, self.len,
                                     window, sinks, status=self.st)

    def check(self, window, sinks):
        torch.cuda.synchronize()
        jca.check_status(self.st)
        kc, vc = self.kc_cpu.clone(), self.vc_cpu.clone()
        for b, p in enumerate(self.lens):
            if p < 0:
                assert bool((self.out[b] == 0).all())
                continue
            s = int(self.off_np[b])
            kc[s + p], vc[s + p] = self.kn_cpu[b], self.vn_cpu[b]
            mask = lh.window_mask(p + 1, window, sinks)[-1:]
            ref, _, _, A = lh.masked(self.q_cpu[b:b + 1], kc[s:s + p + 1], vc[s:s + p + 1], mask, self.scale)
            near(self.out[b:b + 1], ref, (2.0**-8 + 2.0**-11) * A + 2.0**-8 * np.abs(ref) + 1e-30, f"user {b}")
        for got, want in ((self.kc, kc), (self.vc, vc)):     # every other row as it was, bit for bit
            assert torch.equal(got.cpu().view(torch.int16), want.view(torch.int16))


@pytest.mark.parametrize("d", [16, 32, 64, 128])
@pytest.mark.parametrize("H,Hkv", [(2, 2), (8, 2), (16, 1), (40, 2), (3, 1)])
def test_decode_edges(d, H, Hkv):
    lens = [0, 1, 15, 16, 17, -1, 63, 64, 65, 127, 128, 129, 300, 1000]
    for window, sinks in ((1, 0), (2, 5), (64, 4), (100, 0), (1 << 40, 0), (17, 500)):
        b = Decode(lens, [max(n, 0) + 1 + (i % 3) for i, n in enumerate(lens)], H, Hkv, d, seed=d)
        b.run(window, sinks)
        b.check(window, sinks)


@pytest.mark.parametrize("n", [0, 5, 130, 5000, 20000])
def test_decode_one_user(n):
    b = Decode([n], [n + 1], 8, 8, 128, seed=n, idx=torch.int32, spare=0)
    b.run(1 << 20, 0)
    b.check(1 << 20, 0)
    b = Decode([n], [n + 9], 8, 2, 64, seed=n)
    b.run(4000, 4)
    b.check(4000, 4)


def test_decode_strided_rows():
    b = Decode([30, 7, 90], [40, 40, 100], 4, 2, 64, seed=1)
    x = torch.cat([b.q, b.kn, b.vn], 1)
    b.q, b.kn, b.vn = x.split([4, 2, 2], 1)
    b.run(20, 3)
    b.check(20, 3)


def test_decode_follows_the_forward():
    """A row's tokens decoded one after another give the rows of the forward."""
    w = Window([70], 4, 2, 64, seed=5)
    w.forward(16, 3)
    kc, vc = (torch.full((75, 2, 64), float("nan"), dtype=torch.bfloat16, device=dev()) for _ in range(2))
    off, n = torch.tensor([2, 74], device=dev()), torch.zeros(1, dtype=torch.int64, device=dev())
    out, st = torch.empty(1, 4, 64, dtype=torch.bfloat16, device=dev()), jca.new_status(dev())
    rows = []
    for i in range(70):
        jca.jagged_window_decode_fwd(w.q[i:i + 1], w.k[i:i + 1], w.v[i:i + 1], kc, vc, out, off, n, 16, 3, status=st)
        rows.append(out.clone())
        n += 1
    jca.check_status(st)
    w.out = torch.cat(rows)
    w.lse = None
    w.check_forward(16, 3)
    assert torch.equal(kc[2:72], w.k) and torch.equal(vc[2:72], w.v)


def test_decode_bad_users_leave_the_others():
    b = Decode([5, 6, 7], [8, 8, 8], 2, 2, 16, seed=2)
    for off, n, code in (([0, 8, 4, 24], [5, 6, 7], 2), ([0, 8, 16, 28], [5, 6, 7], 2), ([-8, 8, 16, 24], [5, 6, 7], 2),
                         ([0, 8, 16, 24], [5, 8, 7], 1), ([0, 8, 16, 24], [5, -2, 7], 1)):
        b.off, b.len = torch.tensor(off, device=dev()), torch.tensor(n, device=dev())
        st = jca.new_status(dev())
        kc = b.kc.clone()
        out = torch.full_like(b.out, 7.0)
        jca.jagged_window_decode_fwd(b.q, b.kn, b.vn, kc, b.vc, out, b.off, b.len, 4, 1, status=st)
        torch.cuda.synchronize()
        assert int(st.item()) == code
        bad = [u for u in range(3) if not (0 <= off[u] <= off[u + 1] <= 27 and -1 <= n[u] < off[u + 1] - off[u])]
        assert bool((out[bad] == 7.0).all())


def test_decode_captured_twice_and_two_streams():
    """Two graphs over one cache, replayed in turn with the lengths counted on the device, and two
    batches on two streams."""
    a, b = (Decode([5, 600, -1], [40, 700, 3], 8, 2, 64, seed=s) for s in (3, 4))
    graphs = []
    for x in (a, b):
        x.run(200, 2)
        x.check(200, 2)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            x.run(200, 2)
        graphs.append(g)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in graphs]
    for x in (a, b):
        x.out.fill_(float("nan"))
    torch.cuda.synchronize()
    for g, s in zip(graphs, streams):
        with torch.cuda.stream(s):
            g.replay()
    torch.cuda.synchronize()
    for x in (a, b):
        x.check(200, 2)
        # One token further.
        x.len += (x.len >= 0).long()
        torch.cuda.synchronize()
    for x, g in zip((a, b), graphs):
        g.replay()
        torch.cuda.synchronize()
        for u, p in enumerate(x.lens):
            if p >= 0:
                s = int(x.off_np[u])
                x.kc_cpu[s + p], x.vc_cpu[s + p] = x.kn_cpu[u], x.vn_cpu[u]
                x.lens[u] = p + 1
        x.check(200, 2)


def test_decode_many_users_equal_bits():
    rng = np.random.default_rng(8)
    lens = list(rng.integers(-1, 300, 700))
    b = Decode(lens, [int(n) + 2 for n in lens], 8, 2, 128, seed=9)
    b.run(128, 4)
    b.check(128, 4)
    first = b.out.clone()
    b.run(128, 4)
    assert torch.equal(first, b.out)


# ------------------------------------------------------------------------------------------------
# Trees of drafted tokens
# ------------------------------------------------------------------------------------------------

class Tree:
    def __init__(self, counts, hist, H, Hkv, d, seed=0, idx=torch.int64, shape="random", hist_len=None):
        g = torch.Generator().manual_seed(seed)
        rng = np.random.default_rng(seed)
        self.counts, self.hist = counts, hist
        self.use = list(hist if hist_len is None else hist_len)
        N, R = sum(counts), sum(hist) + 5
        self.coff = np.concatenate([[0], np.cumsum(counts)]).astype(np.int64)
        self.hoff = np.concatenate([[0], np.cumsum(hist)]).astype(np.int64)
        self.cpu = [torch.randn(N, h, d, generator=g).to(torch.bfloat16) for h in (H, Hkv, Hkv)]
        self.cache = [torch.randn(R, Hkv, d, generator=g).to(torch.bfloat16) for _ in range(2)]
        used = np.zeros(R, bool)
        for b, n in enumerate(self.use):
            used[self.hoff[b]:self.hoff[b] + n] = True
        for x in self.cache:
            x[~used] = float("nan")
        par = []
        for n in counts:
            i = np.arange(n)
            if shape == "chain":
                par.append(i - 1)
            elif shape == "star":
                par.append(np.full(n, -1))
            else:
                par.append(np.array([rng.integers(-1, t) if t else -1 for t in range(n)], dtype=np.int64))
        self.par = par
        self.parent = torch.tensor(np.concatenate(par) if par else [], dtype=torch.int32, device=dev())
        self.q, self.k, self.v = (x.to(dev()) for x in self.cpu)
        self.hk, self.hv = (x.to(dev()) for x in self.cache)
        self.off, self.ho = (torch.tensor(x, dtype=idx, device=dev()) for x in (self.coff, self.hoff))
        self.hl = None if hist_len is None else torch.tensor(hist_len, dtype=idx, device=dev())
        self.out = torch.full((N, H, d), float("nan"), dtype=torch.bfloat16, device=dev())
        self.scale, self.st = d**-0.5, jca.new_status(dev())

    def run(self, max_cand=None):
        jca.cand_tree_attn_fwd(self.q, self.k, self.v, self.off, self.parent, self.hk, self.hv, self.ho, self.out,
                               max_cand or max(max(self.counts), 1), hist_len=self.hl, status=self.st)

    def check(self):
        torch.cuda.synchronize()
        jca.check_status(self.st)
        for b, n in enumerate(self.counts):
            if n == 0:
                continue
            c, h0 = slice(int(self.coff[b]), int(self.coff[b + 1])), int(self.hoff[b])
            k, v = (torch.cat([x[h0:h0 + self.use[b]], y[c]]) for x, y in zip(self.cache, self.cpu[1:]))
            ref, _, _, A = lh.masked(self.cpu[0][c], k, v, lh.tree_mask(self.par[b], self.use[b]), self.scale)
            near(self.out[c], ref, (2.0**-8 + 2.0**-11) * A + 2.0**-8 * np.abs(ref) + 1e-30, f"user {b}")


@pytest.mark.parametrize("d", [16, 32, 64, 128])
@pytest.mark.parametrize("H,Hkv", [(2, 2), (8, 2), (5, 1), (16, 1), (40, 1)])
def test_tree_edges(d, H, Hkv):
    b = Tree([1, 0, 7, 16, 17, 33, 64, 65, 3], [0, 12, 1, 63, 64, 65, 130, 300, 128], H, Hkv, d, seed=d)
    b.run()
    b.check()


@pytest.mark.parametrize("shape", ["chain", "star", "random"])
def test_tree_large(shape):
    b = Tree([1024, 700], [40, 0], 2, 1, 64, seed=1, shape=shape, idx=torch.int32)
    b.run()
    b.check()


def test_tree_long_history_of_one_user():
    b = Tree([9], [6000], 8, 8, 128, seed=2)
    b.run(64)
    b.check()


def test_tree_regions_with_room():
    b = Tree([5, 12, 4], [100, 70, 40], 8, 4, 128, seed=3, hist_len=[64, 0, 39])
    b.run()
    b.check()


def test_tree_strided_rows_and_graph():
    b = Tree([9, 20], [200, 77], 4, 2, 64, seed=4)
    x = torch.cat([b.q, b.k, b.v], 1)
    b.q, b.k, b.v = x.split([4, 2, 2], 1)
    b.run()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        b.run()
    b.out.fill_(float("nan"))
    graph.replay()
    b.check()


def test_star_tree_is_the_candidate_only_layer():
    b = Tree([40, 3, 100], [90, 500, 17], 4, 4, 64, seed=6, shape="star")
    b.run()
    out = torch.empty_like(b.out)
    st = jca.new_status(dev())
    jca.cand_only_attn_fwd(b.q, b.k, b.v, b.off, b.hk[:607], b.hv[:607], b.ho, out, status=st)
    jca.check_status(st)
    b.check()
    torch.testing.assert_close(b.out.float(), out.float(), atol=3e-2, rtol=2.0**-6)


@pytest.mark.parametrize("B,H,Hkv,lens", [(600, 2, 2, True), (257, 8, 8, False), (300, 48, 2, True), (450, 1, 1, False)])
def test_tree_many_users_in_any_order(B, H, Hkv, lens):
    """More blocks than run at once: users are then taken by length, in groups of 256."""
    rng = np.random.default_rng(B)
    hist = [int(x) for x in np.floor(rng.lognormal(3.0, 1.5, B)).clip(0, 2000)]
    hist[5], hist[B - 1], hist[B // 2] = 0, 700, 0
    use = [int(rng.integers(0, n + 1)) for n in hist] if lens else None
    b = Tree([int(x) for x in rng.integers(0, 6, B)], hist, H, Hkv, 32, seed=B, hist_len=use)
    b.run()
    b.check()
    first = b.out.clone()
    b.run()
    assert torch.equal(first, b.out)


def test_tree_many_users_with_a_bad_one():
    """Lengths that mean nothing change no other user's place."""
    n = 500
    for name, at, x, code in (("hl", 300, -5, 1), ("hl", 7, 1 << 40, 1), ("ho", n, 1 << 40, 2)):
        b = Tree([2] * n, [10] * n, 2, 2, 16, seed=1, hist_len=[10] * n)
        want = torch.empty_like(b.out)
        b.run()
        b.check()
        want.copy_(b.out)
        user = at if name == "hl" else n - 1
        getattr(b, name)[at] = x
        b.out.fill_(7.0)
        b.run()
        torch.cuda.synchronize()
        assert int(b.st.item()) == code
        assert bool((b.out[2 * user:2 * user + 2] == 7.0).all())
        rest = torch.ones(2 * n, dtype=torch.bool, device=dev())
        rest[2 * user:2 * user + 2] = False
        # Right, or not written; head by head, since a user's heads see the status at different times.
        same = (b.out == want).all(2) | (b.out == 7.0).all(2)
        assert bool(same[rest].all())


def test_tree_bad_users_leave_the_others():
    def code(**kw):
        b = Tree([4, 6, 3], [20, 30, 10], 2, 2, 16, seed=5, hist_len=[20, 30, 10])
        b.out.fill_(7.0)
        for name, (i, x) in kw.items():
            getattr(b, name)[i] = x
        b.run(6)
        torch.cuda.synchronize()
        assert bool((b.out[4:10] == 7.0).all())
        return int(b.st.item())

    assert code(parent=(4, 0)) == 8            # its own parent
    assert code(parent=(6, 3)) == 8            # a later token
    assert code(parent=(9, -2)) == 8
    assert code(hl=(1, 31)) == 1
    assert code(hl=(1, -1)) == 1
    assert code(ho=(2, 200)) == 2
    assert code(off=(1, 11)) in (2, 8)         # falling offsets, and a first run of 11: either wins
    b = Tree([4, 6, 3], [20, 30, 10], 2, 2, 16, seed=5)
    b.out.fill_(7.0)
    b.run(5)                                   # a run longer than max_cand
    torch.cuda.synchronize()
    assert int(b.st.item()) == 8 and bool((b.out[4:10] == 7.0).all())


# ------------------------------------------------------------------------------------------------
# Rotary positions with several axes
# ------------------------------------------------------------------------------------------------

def _rope_check(x, got, pos, sections, per_axis, sign, what, base=10000.0):
    ref = lh.rope_axes(x, pos, sections, base, per_axis, sign)
    a = np.abs(lh.f64(x))
    half = a.shape[2] // 2
    both = np.concatenate([a[..., :half] + a[..., half:]] * 2, -1)
    near(got, ref, HALF[x.dtype] * np.abs(ref) + 2.0**-22 * both + 1e-30, what)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("d,sections", [(16, [8]), (16, [3, 2, 2]), (32, [0, 16]), (64, [9, 10, 10]),
                                        (128, [16, 24, 24]), (128, [1, 0, 20, 30]), (128, [0])])
def test_rope_axes(dtype, d, sections):
    g = torch.Generator().manual_seed(d)
    T, A = 77, len(sections)
    q, k = torch.randn(T, 5, d, generator=g).to(dtype), torch.randn(T, 2, d, generator=g).to(dtype)
    pos = torch.randint(-40, 5000, (T, A), generator=g)
    pos[:, -1] = torch.randint(1 << 30, 1 << 31, (T,), generator=g) - (1 << 20)    # seconds since an epoch
    for per_axis in (False, True):
        for idx in (torch.int32, torch.int64):
            for fn, sign in ((jca.jca_rope_axes_fwd, 1.0), (jca.jca_rope_axes_bwd, -1.0)):
                qo, ko = torch.empty_like(q, device=dev()), torch.empty_like(k, device=dev())
                p = pos.to(idx).to(dev())
                fn(q.to(dev()), k.to(dev()), qo, ko, p, sections, per_axis=per_axis)
                _rope_check(q, qo, pos, sections, per_axis, sign, "q")
                _rope_check(k, ko, pos, sections, per_axis, sign, "k")


def test_rope_axes_in_place_strided_and_alone():
    g = torch.Generator().manual_seed(1)
    x = torch.randn(200, 8, 64, generator=g).to(torch.bfloat16)
    pos = torch.randint(0, 4096, (200, 2), generator=g)
    y = x.to(dev())
    q, k = y[:, :4], y[:, 4:6]
    jca.jca_rope_axes_fwd(q, k, q, k, pos.to(dev()), [20, 8])
    _rope_check(x[:, :4], q, pos, [20, 8], False, 1.0, "q")
    _rope_check(x[:, 4:6], k, pos, [20, 8], False, 1.0, "k")
    assert torch.equal(y[:, 6:].cpu(), x[:, 6:])
    alone = torch.empty(200, 4, 64, dtype=torch.bfloat16, device=dev())
    jca.jca_rope_axes_fwd(x.to(dev())[:, :4], None, alone, None, pos.to(dev()), [20, 8])
    assert torch.equal(alone, q)


def test_rope_one_axis_is_jca_apply_rope():
    g = torch.Generator().manual_seed(2)
    x = torch.randn(300, 3, 128, generator=g).to(torch.bfloat16).to(dev())
    pos = torch.randint(0, 4096, (300,), generator=g).to(torch.int32).to(dev())
    a, b = torch.empty_like(x), torch.empty_like(x)
    jca.jca_apply_rope(x, a, pos)
    jca.jca_rope_axes_fwd(x, None, b, None, pos, [64])
    torch.testing.assert_close(a.float(), b.float(), atol=1e-5, rtol=2.0**-7)


def test_rope_other_pairs_hold_anything():
    """Pairs past the sections are copied bit for bit, whatever they hold."""
    x = torch.randn(9, 2, 32).to(torch.bfloat16)
    x[..., 10:16] = float("inf")
    x[..., 26:32] = float("nan")
    y = torch.empty_like(x, device=dev())
    jca.jca_rope_axes_fwd(x.to(dev()), None, y, None, torch.arange(18, device=dev()).view(9, 2), [5, 5])
    got = y.cpu()
    keep = list(range(10, 16)) + list(range(26, 32))
    assert torch.equal(got[..., keep].view(torch.int16), x[..., keep].view(torch.int16))
    assert bool(torch.isfinite(got[..., :10].float()).all())


# ------------------------------------------------------------------------------------------------
# Together
# ------------------------------------------------------------------------------------------------

def test_layer_of_a_training_step_and_its_serving():
    """Rotation, windowed attention, its gradient and the rotation's, against the composed fp64
    formulas; then the cache that serving builds from the same rows: prefill, decoded tokens, drafts."""
    H, Hkv, d, W, S, sections = 4, 2, 64, 24, 2, [12, 10, 10]
    lengths = [60, 9, 131]
    b = Window(lengths, H, Hkv, d, seed=20)
    g = torch.Generator().manual_seed(3)
    pos = torch.randint(0, 3000, (b.T, 3), generator=g)
    p = pos.to(dev())
    qr, kr = torch.empty_like(b.q), torch.empty_like(b.k)
    jca.jca_rope_axes_fwd(b.q, b.k, qr, kr, p, sections)
    q0, k0 = b.q_cpu, b.k_cpu
    b.q, b.k, b.q_cpu, b.k_cpu = qr, kr, qr.cpu(), kr.cpu()
    _rope_check(q0, qr, pos, sections, False, 1.0, "q")
    b.forward(W, S)
    b.check_forward(W, S)
    b.backward(W, S)
    b.check_backward(W, S)
    dq, dk = torch.empty_like(b.q), torch.empty_like(b.k)
    jca.jca_rope_axes_bwd(b.grads[0], b.grads[1], dq, dk, p, sections)
    _rope_check(b.grads[0].cpu(), dq, pos, sections, False, -1.0, "dq")
    _rope_check(b.grads[1].cpu(), dk, pos, sections, False, -1.0, "dk")
    # serving: every row but its last token is prefilled, the last is decoded
    b.forward(W, S)
    n = torch.tensor([x - 1 for x in lengths], device=dev())
    last = (b.off[1:] - 1)
    kc, vc = b.k.clone(), b.v.clone()
    kc[last], vc[last] = float("nan"), float("nan")
    out, st = torch.empty(3, H, d, dtype=torch.bfloat16, device=dev()), jca.new_status(dev())
    jca.jagged_window_decode_fwd(b.q[last], b.k[last], b.v[last], kc, vc, out, b.off, n, W, S, status=st)
    jca.check_status(st)
    assert torch.equal(kc, b.k) and torch.equal(vc, b.v)
    torch.testing.assert_close(out.float(), b.out[last].float(), atol=3e-2, rtol=2.0**-6)
    # drafts over the same cache: a chain is a causal continuation of it
    t = Tree([5, 5, 5], lengths, H, Hkv, d, seed=21, shape="chain")
    t.hk[: b.T], t.hv[: b.T] = kc, vc
    t.cache[0][: b.T], t.cache[1][: b.T] = kc.cpu(), vc.cpu()
    t.run()
    t.check()


# ------------------------------------------------------------------------------------------------
# Large offsets, threads
# ------------------------------------------------------------------------------------------------

def test_caches_beyond_32_bit_offsets():
    """Users at both ends of a cache of more than 2^31 elements, for one token and for trees."""
    H, d, n, last = 8, 128, 300, 2**21 + 5000
    R = last + n + 1
    assert last * H * d > 2**31
    g = torch.Generator().manual_seed(1)
    kc, vc = (torch.empty(R, H, d, dtype=torch.bfloat16, device=dev()) for _ in range(2))
    kh, vh = (torch.randn(2, n, H, d, generator=g).to(torch.bfloat16) for _ in range(2))
    for c, x in ((kc, kh), (vc, vh)):
        c[:n], c[last:last + n] = x[0].to(dev()), x[1].to(dev())
    q, k, v = (torch.randn(6, H, d, generator=g).to(torch.bfloat16) for _ in range(3))
    st = jca.new_status(dev())
    off = torch.tensor([0, last, R], device=dev())
    used = torch.tensor([n, n], device=dev())
    parent = torch.tensor([-1, 0, 0, -1, 0, 1], dtype=torch.int32, device=dev())
    out = torch.empty(6, H, d, dtype=torch.bfloat16, device=dev())
    jca.cand_tree_attn_fwd(q.to(dev()), k.to(dev()), v.to(dev()), torch.tensor([0, 3, 6], device=dev()), parent, kc, vc,
                           off, out, 3, hist_len=used, status=st)
    jca.check_status(st)
    for b, par in enumerate(([-1, 0, 0], [-1, 0, 1])):
        t = slice(3 * b, 3 * b + 3)
        ref, _, _, A = lh.masked(q[t], torch.cat([kh[b], k[t]]), torch.cat([vh[b], v[t]]), lh.tree_mask(par, n), d**-0.5)
        near(out[t], ref, (2.0**-8 + 2.0**-11) * A + 2.0**-8 * np.abs(ref), f"tree {b}")
    one = torch.empty(2, H, d, dtype=torch.bfloat16, device=dev())
    jca.jagged_window_decode_fwd(q[:2].to(dev()), k[:2].to(dev()), v[:2].to(dev()), kc, vc, one, off, used, 100, 5,
                                 status=st)
    jca.check_status(st)
    mask = lh.window_mask(n + 1, 100, 5)[-1:]
    for b, at in enumerate((n, last + n)):
        assert torch.equal(kc[at].cpu(), k[b]) and torch.equal(vc[at].cpu(), v[b])
        ref, _, _, A = lh.masked(q[b:b + 1], torch.cat([kh[b], k[b:b + 1]]), torch.cat([vh[b], v[b:b + 1]]), mask, d**-0.5)
        near(one[b:b + 1], ref, (2.0**-8 + 2.0**-11) * A + 2.0**-8 * np.abs(ref), f"token {b}")


def test_rope_rows_beyond_32_bit_offsets():
    T, H, d = 2**21 + 1001, 8, 128
    g = torch.Generator(device=dev()).manual_seed(2)
    q = torch.empty(T, H, d, dtype=torch.bfloat16, device=dev()).normal_(generator=g)
    pos = torch.randint(-1000, 1 << 40, (T, 2), generator=g, device=dev())
    ends = [slice(0, 40), slice(T - 40, T)]
    kept = [q[r].cpu() for r in ends]
    jca.jca_rope_axes_fwd(q, None, q, None, pos, [40, 24])
    for r, x in zip(ends, kept):
        ref = lh.rope_axes(x, pos[r].cpu(), [40, 24])
        a = np.abs(lh.f64(x))
        both = np.concatenate([a[..., :64] + a[..., 64:]] * 2, -1)
        # The angle is off by 2^40 2^-61 turns at most, 2^-18 of a radian.
        near(q[r], ref, 2.0**-8 * np.abs(ref) + (2.0**-22 + 2.0**-18) * both, f"rows {r}")


def test_calls_from_two_threads():
    """Each thread its own stream, batch and buffers; every operator, first calls included."""
    import threading
    wrong = []

    def work(seed):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                w = Window([90, 200 + seed], 4, 2, 32, seed=seed)
                d = Decode([50, 7], [60, 9], 4, 2, 32, seed=seed)
                t = Tree([4, 9], [30, 70], 4, 2, 32, seed=seed)
                for _ in range(4):
                    w.forward(40, 2)
                    d.run(30, 2)
                    t.run()
                    w.check_forward(40, 2)
                    w.backward(40, 2)
                    w.check_backward(40, 2)
                    d.check(30, 2)
                    t.check()
        except BaseException as e:                                  # noqa: BLE001
            wrong.append(e)

    torch.cuda.synchronize()
    threads = [threading.Thread(target=work, args=(s,)) for s in (21, 22)]
    for x in threads:
        x.start()
    for x in threads:
        x.join()
    assert not wrong, wrong


def test_longest_list_of_keys():
    """A list of 2^31 - 2 keys, the longest that is accepted: one token and one draft over a history of
    which four rows, the first and the last of the cache among them, hold nearly all the weight."""
    d, R = 16, 2**31 - 2
    torch.cuda.empty_cache()
    if torch.cuda.mem_get_info()[0] < 4 * R * d + (4 << 30):
        pytest.skip("two caches of 2^35 elements need 138 GB")
    kc, vc = (torch.zeros(R, 1, d, dtype=torch.bfloat16, device=dev()) for _ in range(2))
    g = torch.Generator().manual_seed(3)
    rows = [0, 2**30 + 17, R - 2]
    v = torch.randn(5, 1, d, generator=g).to(torch.bfloat16)
    for i, r in enumerate(rows):
        kc[r], vc[r] = 10.0, v[i].to(dev())
    q = torch.ones(1, 1, d, dtype=torch.bfloat16, device=dev())
    kn, out, st = 10.0 * q, torch.full_like(q, float("nan")), jca.new_status(dev())
    off, n = torch.tensor([0, R], device=dev()), torch.tensor([R - 1], device=dev())
    # Scores 40 for the four, 0 for the rest, whose values are 0.
    heavy = np.exp(40.0)

    def check(x):
        want = heavy * lh.f64(x).sum(0) / (len(x) * heavy + R - len(x))
        A = heavy * np.abs(lh.f64(x)).sum(0) / (len(x) * heavy)
        near(out[0], want, (2.0**-8 + 2.0**-11) * A + 2.0**-8 * np.abs(want), f"{len(x)} rows")

    jca.jagged_window_decode_fwd(q, kn, v[3:4].to(dev()), kc, vc, out, off, n, 1 << 40, 0, status=st)
    jca.check_status(st)
    check(v[:4])
    assert bool((kc[R - 1] == 10.0).all()) and torch.equal(vc[R - 1].cpu(), v[3])
    out.fill_(float("nan"))
    jca.cand_tree_attn_fwd(q, kn, v[4:].to(dev()), torch.tensor([0, 1], device=dev()),
                           torch.tensor([-1], dtype=torch.int32, device=dev()), kc, vc, off, out, 1, status=st)
    jca.check_status(st)
    check(v)                                       # the new row of the cache among them
    del kc, vc
    torch.cuda.empty_cache()


# ------------------------------------------------------------------------------------------------
# Reach of a real token that is not finite
# ------------------------------------------------------------------------------------------------

def _tile_reads(off, window, sinks):
    """[T, T]: row i lies in a query tile that reads row r, by include/jca.h."""
    T = int(off[-1])
    start = np.repeat(off[:-1], np.diff(off))
    r, got = np.arange(T), np.zeros((T, T), bool)
    for a in range(0, T, 128):
        s = int(start[a])
        got[a:a + 128] = (r >= max(s, a - window + 1) - 127) & (r < a + 128)
        if sinks:
            got[a:a + 128] |= (r >= s - 127) & (r < s + sinks + 127)
    return got


def _tile_queries(off, window, sinks):
    """[T, T]: query row r is among those that key row j's gradients are formed with."""
    T = int(off[-1])
    end = np.repeat(off[1:], np.diff(off))
    r, got = np.arange(T), np.zeros((T, T), bool)
    for a in range(0, T, 128):
        last = min(a + 128, T) - 1
        got[a:a + 128] = (r >= a) & (r < min(int(end[last]), a + 127 + window) + 63)
    for s, e in zip(off[:-1], off[1:]):
        if e - s > window:
            got[s:min(s + sinks, e)] |= (r >= s + window - 63) & (r < e + 63)
    return got


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("window,sinks", [(1024, 0), (1024, 3), (70, 0), (1, 5), (130, 100)])
def test_window_reach_of_a_token_that_is_not_finite(window, sinks, d):
    """One row of one user holds NaN or Inf. All rows beyond the stated reach are as without it, bit for
    bit, and the rows that see it are not finite."""
    b = Window([100, 1000, 60, 7, 300], 2, 1, d, seed=30)
    sees = np.zeros((b.T, b.T), bool)
    for r, mask in b.users(window, sinks):
        sees[r, r] = mask
    reads, queries = _tile_reads(b.off_np, window, sinks), _tile_queries(b.off_np, window, sinks)
    assert (reads | ~sees).all() and (queries | ~sees.T).all()
    own = np.eye(b.T, dtype=bool)

    def forward(**kw):
        x = {**dict(q=b.q, k=b.k, v=b.v), **kw}
        out, lse = torch.empty_like(b.q), torch.empty(b.T, 2, device=dev())
        jca.jagged_window_attn_fwd(x["q"], x["k"], x["v"], out, b.off, window, sinks, lse=lse, status=b.st)
        return out, lse

    def backward(**kw):
        x = {**dict(q=b.q, k=b.k, v=b.v, dout=b.dout), **kw}
        grads = [torch.empty_like(t) for t in (b.q, b.k, b.v)]
        jca.jagged_window_attn_bwd(x["q"], x["k"], x["v"], out, x["dout"], lse, *grads, b.off, window, sinks,
                                   status=b.st)
        return grads

    out, lse = forward()
    clean = [out, lse] + backward()
    jca.check_status(b.st)
    none = np.zeros_like(own)
    # Row i of (out, lse, dq, dk, dv) may differ for a bad row r of the input.
    reach = dict(q=(own, own, own, queries, queries), k=(sees, sees, reads, own, own),
                 v=(reads, none, sees, own, none), dout=(none, none, own, queries, queries))
    for name, spread in reach.items():
        for r in (0, 50, 99, 100, 127, 128, 700, 1099, 1100, 1160, 1166, 1167, b.T - 1):
            bad = getattr(b, name).clone()
            bad[r] = float("nan") if r % 2 else float("inf")
            got = list(forward(**{name: bad}) if name != "dout" else (out, lse)) + backward(**{name: bad})
            jca.check_status(b.st)
            for what, x, y, where in zip(("out", "lse", "dq", "dk", "dv"), got, clean, spread):
                keep = torch.tensor(~where[:, r], device=dev())
                assert torch.equal(x[keep], y[keep]), f"{name} {r}: {what}"
            if name == "v":
                seen = torch.tensor(sees[:, r], device=dev())
                assert not bool(torch.isfinite(got[0][seen].float()).any())


def test_cache_rows_that_are_not_finite_stay_with_their_user():
    """Trees: a bad k or q of a drafted token only in the rows that see it, a bad v only in its run, a
    bad history row only in its user. One token: rows it does not see hold NaN."""
    for H, Hkv, d in ((2, 2, 64), (8, 2, 128), (40, 2, 32)):
        b = Tree([5, 70, 9], [30, 130, 65], H, Hkv, d, seed=40)
        b.run()
        b.check()
        clean = b.out.clone()
        for name, at in (("q", 20), ("k", 20), ("v", 20), ("v", 74), ("hk", 100), ("hv", 31)):
            x = getattr(b, name)
            kept = x[at].clone()
            x[at] = float("nan")
            b.out.fill_(7.0)
            b.run()
            jca.check_status(b.st)
            x[at] = kept
            hit = np.zeros(84, bool)
            if name in "qk":
                hit[5:75] = lh.tree_mask(b.par[1], 0)[:, 15] if name == "k" else np.arange(70) == 15
            else:
                hit[5:75] = True
            keep = torch.tensor(~hit, device=dev())
            assert torch.equal(b.out[keep], clean[keep]), (name, at)
        c = Decode([50, 90, 3], [60, 90 + 1, 9], H, Hkv, d, seed=41)
        c.run(20, 4)
        c.check(20, 4)
        clean = c.out.clone()
        for x in (c.kc, c.vc):
            x[4:31] = float("nan")                 # behind user 0's first tokens, before its window
        c.run(20, 4)
        assert torch.equal(c.out, clean)
        c.kc[60 + 80], c.vc[60 + 81] = float("nan"), float("inf")
        c.run(20, 4)
        jca.check_status(c.st)
        assert torch.equal(c.out[[0, 2]], clean[[0, 2]])
        assert not bool(torch.isfinite(c.out[1].float()).any())


# ------------------------------------------------------------------------------------------------
# Users with bad data beside good ones: nothing of theirs is written, nothing of the others is wrong
# ------------------------------------------------------------------------------------------------

def _right_or_unwritten(got, want, rows, fill, what):
    """Head by head, since the blocks of a user see the status at different times."""
    same = (got == want).all(2) | (got == fill).all(2)
    assert bool(same[rows].all()), what


def _bits(x):
    return x.view(torch.int16)


@pytest.mark.parametrize("H,Hkv,d", [(2, 2, 16), (16, 2, 128), (40, 1, 64)])
def test_decode_bad_users_write_nothing(H, Hkv, d):
    """A cache_len that fills its region would append to the next user's first row."""
    rng = np.random.default_rng(H)
    for B in (3, 400):
        lens = [int(x) for x in rng.integers(0, 90, B)]
        lens[:3] = [5, 8, 7]
        caps = [n + 1 + int(x) for n, x in zip(lens, rng.integers(0, 3, B))]
        b = Decode(lens, caps, H, Hkv, d, seed=B)
        kc, vc = b.kc.clone(), b.vc.clone()
        for name, at, x, code in (("len", 1, caps[1], 1), ("len", 1, caps[1] + 3, 1), ("len", 0, -2, 1),
                                  ("len", B - 1, 1 << 40, 1), ("off", 0, -8, 2), ("off", B, 1 << 40, 2),
                                  ("off", B, 0, 2)):
            bad = at if name == "len" else min(at, B - 1)
            # The batch with an empty slot in the bad user's place.
            b.len[bad], kept = -1, int(b.len[bad])
            b.kc.copy_(kc)
            b.vc.copy_(vc)
            b.st.zero_()
            b.run(30, 2)
            jca.check_status(b.st)
            want, wk, wv = b.out.clone(), b.kc.clone(), b.vc.clone()
            b.len[bad] = kept
            held = int(getattr(b, name)[at])
            getattr(b, name)[at] = x
            b.kc.copy_(kc)
            b.vc.copy_(vc)
            b.out.fill_(7.0)
            b.run(30, 2)
            torch.cuda.synchronize()
            what = f"B={B} {name}[{at}]={x}"
            assert int(b.st.item()) == code, what
            assert bool((b.out[bad] == 7.0).all()), what
            rest = torch.arange(B, device=dev()) != bad
            _right_or_unwritten(b.out, want, rest, 7.0, what)
            # Cache rows: as before, or with the new token of a good user, head by head.
            for got, old, new in ((b.kc, kc, wk), (b.vc, vc, wv)):
                same = (_bits(got) == _bits(old)).all(2) | (_bits(got) == _bits(new)).all(2)
                assert bool(same.all()), what
            getattr(b, name)[at] = held


def test_decode_falling_offsets_write_nothing_of_their_user():
    """Users 0 and 2 are good; the region of user 2 then starts inside that of user 0."""
    b = Decode([5, 6, 7], [8, 8, 8], 2, 2, 16, seed=2)
    b.off = torch.tensor([0, 8, 4, 24], device=dev())
    kc, vc = b.kc.clone(), b.vc.clone()
    b.out.fill_(7.0)
    b.run(4, 1)
    torch.cuda.synchronize()
    assert int(b.st.item()) == 2 and bool((b.out[1] == 7.0).all())
    for u, first in ((0, 0), (2, 4)):
        p = b.lens[u]
        k, v = (torch.cat([x[first:first + p], y[u:u + 1]]) for x, y in ((b.kc_cpu, b.kn_cpu), (b.vc_cpu, b.vn_cpu)))
        mask = lh.window_mask(p + 1, 4, 1)[-1:]
        ref, _, _, A = lh.masked(b.q_cpu[u:u + 1], k, v, mask, b.scale)
        for h in range(2):
            if bool((b.out[u, h] == 7.0).all()):
                continue
            near(b.out[u:u + 1, h], ref[:, h], (2.0**-8 + 2.0**-11) * A[:, h] + 2.0**-8 * np.abs(ref[:, h]) + 1e-30,
                 f"user {u}")
    for got, old, new in ((b.kc, kc, b.kn), (b.vc, vc, b.vn)):
        want = old.clone()
        want[5], want[11] = new[0], new[2]
        same = (_bits(got) == _bits(old)).all(2) | (_bits(got) == _bits(want)).all(2)
        assert bool(same.all())


@pytest.mark.parametrize("H,Hkv,d", [(2, 2, 16), (8, 2, 128), (40, 1, 64)])
def test_tree_bad_users_write_nothing(H, Hkv, d):
    n = [4, 6, 3]
    for name, at, x, bad, code in (("parent", 4, 0, [1], 8), ("parent", 6, 3, [1], 8), ("parent", 9, -2, [1], 8),
                                   ("parent", 0, 1 << 30, [0], 8), ("hl", 1, 31, [1], 1), ("hl", 1, -1, [1], 1),
                                   ("ho", 3, 1 << 40, [2], 2), ("ho", 0, -1, [0], 2), ("off", 1, 11, [0, 1], None),
                                   ("off", 0, 1, [0], 2), ("off", 3, 14, [2], 2), ("off", 1, -5, [0, 1], 2)):
        b = Tree(n, [20, 30, 10], H, Hkv, d, seed=5, hist_len=[20, 30, 10])
        b.run(6)
        b.check()
        want = b.out.clone()
        getattr(b, name)[at] = x
        b.out.fill_(7.0)
        b.run(6)
        torch.cuda.synchronize()
        what = f"{name}[{at}]={x}"
        assert int(b.st.item()) in ((2, 8) if code is None else (code,)), what
        rows = torch.zeros(13, dtype=torch.bool, device=dev())
        for u in bad:
            rows[b.coff[u]:b.coff[u + 1]] = True
        assert bool((b.out[rows] == 7.0).all()), what
        _right_or_unwritten(b.out, want, ~rows, 7.0, what)


# ------------------------------------------------------------------------------------------------
# Workspace of the gradients
# ------------------------------------------------------------------------------------------------

@pytest.mark.parametrize("lengths,window,sinks", [
    ([41] * 120, 40, 3),                 # every user one row longer than the window
    ([2] * 1500, 1, 2), ([1, 2] * 400, 1, 128), ([40, 41] * 60, 40, 5), ([3000], 1, 4),
    ([300, 0, 513, 2, 256, 257, 90], 256, 7), ([255, 258, 511, 514] * 3, 1, 1), ([20] * 50, 20, 9),
    ([5, 900, 5], 904, 3), ([5, 900, 5], 910, 3), ([257] * 40, 255, 128)])
def test_window_gradient_in_the_workspace_of_its_window(lengths, window, sinks):
    """The size for the window is enough: memory behind it stays as it was, and the gradients equal
    those with the size for every window."""
    b = Window(lengths, 4, 2, 32, seed=50)
    sizes = [jca.jca_window_bwd_workspace_bytes(len(lengths), b.T, 4, 2, 32, sinks, *w) for w in ((window,), ())]
    assert sizes[0] <= sizes[1]
    grads = []
    for n in sizes:
        ws = torch.full((n + 65536,), 93, dtype=torch.uint8, device=dev())
        grads.append([x.clone() for x in b.backward(window, sinks, workspace=ws[:n])])
        torch.cuda.synchronize()
        assert bool((ws[n:] == 93).all())
    b.check_backward(window, sinks)
    for x, y in zip(*grads):
        assert torch.equal(x, y)
    with pytest.raises(jca.JcaError):
        b.backward(window, sinks, workspace=torch.empty(sizes[0] - 1, dtype=torch.uint8, device=dev()))


def test_window_gradient_of_a_key_that_very_many_rows_see():
    """A key tile's work of 2.9 million steps, over 2 s: no wait for it gives up. Every query head holds the
    same query, so that the gradients are those of one head for the heads' summed dO."""
    T, H, d = 4096, 45000, 16
    torch.cuda.empty_cache()
    if torch.cuda.mem_get_info()[0] < 6 * 2 * T * H * d + 3 * 4 * T * H + (8 << 30):
        pytest.skip("needs 45 GB")
    g = torch.Generator(device=dev()).manual_seed(9)
    one, k, v = (torch.randn(T, 1, d, generator=g, device=dev()).to(torch.bfloat16) for _ in range(3))
    off, st = torch.tensor([0, T], device=dev()), jca.new_status(dev())
    out1, lse1 = torch.empty_like(one), torch.empty(T, 1, device=dev())
    jca.jagged_window_attn_fwd(one, k, v, out1, off, T, 0, lse=lse1, status=st)
    q, out, lse = (x.expand(T, H, *x.shape[2:]).contiguous() for x in (one, out1, lse1))
    dout = torch.empty_like(q).normal_(generator=g)
    dq, dk, dv = (torch.full_like(x, float("nan")) for x in (q, k, v))
    jca.jagged_window_attn_bwd(q, k, v, out, dout, lse, dq, dk, dv, off, T, 0, status=st)
    jca.check_status(st)
    assert bool(torch.isfinite(dq.sum(1, dtype=torch.float32)).all())
    q1, k1, v1, o1 = (x[:, 0].double() for x in (one, k, v, out1))
    P = torch.exp(d**-0.5 * q1 @ k1.T - lse1.double()).tril()
    total, spread = dout.sum(1, dtype=torch.float64), dout.abs().sum(1, dtype=torch.float64)
    dS = P * (total @ v1.T - (total * o1).sum(1, keepdim=True))
    # |dS| of a head is at most P (|dO| |v| + |dO| |O|); the factors are those of the other gradients.
    most = P * (spread @ v1.abs().T + (spread * o1.abs()).sum(1, keepdim=True))
    for name, got, ref, terms in (("dv", dv, P.T @ total, P.T @ spread),
                                  ("dk", dk, d**-0.5 * dS.T @ q1, d**-0.5 * most.T @ q1.abs())):
        tol = (2.0**-8 + 2.0**-11) * terms + 2.0**-8 * ref.abs()
        near(got[:, 0], ref.cpu().numpy(), tol.cpu().numpy(), name)
    mask = lh.window_mask(T, T, 0)
    for h in (0, H - 1):
        (x, _, _), (tq, _, _) = lh.gradients(one, k, v, dout[:, h:h + 1], mask, d**-0.5)
        near(dq[:, h:h + 1], x, 2.0**-8 * tq[0] + 2.0**-11 * tq[1] + 2.0**-8 * np.abs(x) + 1e-30, f"dq {h}")


@pytest.mark.parametrize("window,sinks", [(1 << 40, 0), (4090, 4), (64, 4)])
def test_window_gradient_of_long_sums(window, sinks):
    """dK and dV of one key head over 8,192 query heads, all terms of dV of one sign: up to 33 million
    products to a sum. In the tensor core's accumulators alone dV came out 3 % small."""
    T, H, d = 4096, 8192, 16
    torch.cuda.empty_cache()
    g = torch.Generator(device=dev()).manual_seed(10)
    one, k, v = (torch.randn(T, 1, d, generator=g, device=dev()).to(torch.bfloat16) for _ in range(3))
    off, st = torch.tensor([0, T], device=dev()), jca.new_status(dev())
    out1, lse1 = torch.empty_like(one), torch.empty(T, 1, device=dev())
    jca.jagged_window_attn_fwd(one, k, v, out1, off, window, sinks, lse=lse1, status=st)
    q, out, lse = (x.expand(T, H, *x.shape[2:]).contiguous() for x in (one, out1, lse1))
    dout = torch.empty_like(q).normal_(generator=g).abs_()
    dq, dk, dv = (torch.full_like(x, float("nan")) for x in (q, k, v))
    jca.jagged_window_attn_bwd(q, k, v, out, dout, lse, dq, dk, dv, off, window, sinks, status=st)
    jca.check_status(st)
    mask = torch.tensor(lh.window_mask(T, window, sinks), device=dev())
    q1, k1, v1, o1 = (x[:, 0].double() for x in (one, k, v, out1))
    P = torch.where(mask, torch.exp(d**-0.5 * q1 @ k1.T - lse1.double()), 0.0)
    total = dout.sum(1, dtype=torch.float64)
    # All terms of dV are positive: P is rounded to bf16 (2^-8), scores and statistics are fp32 (2^-11),
    # the accumulators are cut at most 2^14 times at 2^-23 of the sum (2^-9), the result is rounded.
    ref = P.T @ total
    near(dv[:, 0], ref.cpu().numpy(), (2 * 2.0**-8 + 2.0**-11 + 2.0**-9) * ref.cpu().numpy(), "dv")
    dS = P * (total @ v1.T - (total * o1).sum(1, keepdim=True))
    most = P * (total @ v1.abs().T + (total * o1.abs()).sum(1, keepdim=True))
    ref, terms = d**-0.5 * dS.T @ q1, d**-0.5 * most.T @ q1.abs()
    near(dk[:, 0], ref.cpu().numpy(), ((2.0**-8 + 2.0**-11 + 2.0**-9) * terms + 2.0**-8 * ref.abs()).cpu().numpy(), "dk")
    assert bool(torch.isfinite(dq.sum(1, dtype=torch.float32)).all())


def test_window_rows_that_see_very_many_keys():
    """One user of 600,000 rows: dQ of the last rows and dK, dV of the first are sums over all of them."""
    T, d = 600_000, 16
    g = torch.Generator(device=dev()).manual_seed(11)
    q, k, v, do = (torch.randn(T, 1, d, generator=g, device=dev()).to(torch.bfloat16) for _ in range(4))
    off, st = torch.tensor([0, T], device=dev()), jca.new_status(dev())
    out, lse = torch.empty_like(q), torch.empty(T, 1, device=dev())
    jca.jagged_window_attn_fwd(q, k, v, out, off, T, 0, lse=lse, status=st)
    jca.check_status(st)
    grads = [torch.full_like(x, float("nan")) for x in (q, k, v)]
    jca.jagged_window_attn_bwd(q, k, v, out, do, lse, *grads, off, T, 0, status=st)
    jca.check_status(st)
    q1, k1, v1, o1, do1 = (x[:, 0].double() for x in (q, k, v, out, do))
    scale, D, E = d**-0.5, (do1 * o1).sum(1, keepdim=True), (do1 * o1).abs().sum(1, keepdim=True)
    j = torch.arange(T, device=dev())
    last = torch.tensor([T - 1, T - 100, T // 2, 300_001], device=dev())
    S = scale * q1[last] @ k1.T
    P = torch.where(j[None] <= last[:, None], torch.exp(S - S.amax(1, keepdim=True)), 0.0)
    P /= P.sum(1, keepdim=True)
    ref, A = P @ v1, P @ v1.abs()
    near(out[last, 0], ref.cpu().numpy(), ((2.0**-8 + 2.0**-11) * A + 2.0**-8 * ref.abs()).cpu().numpy(), "out")
    dS = P * (do1[last] @ v1.T - D[last])
    soft, hard = dS.abs() + P * E[last], P * (do1[last].abs() @ v1.abs().T + D[last].abs() + E[last])
    ref = scale * dS @ k1
    tol = scale * (2.0**-8 * soft + 2.0**-11 * hard) @ k1.abs() + 2.0**-8 * ref.abs()
    near(grads[0][last, 0], ref.cpu().numpy(), tol.cpu().numpy(), "dq")
    first = torch.tensor([0, 1, 127, 128, T // 2], device=dev())
    P = torch.where(j[:, None] >= first[None], torch.exp(scale * q1 @ k1[first].T - lse.double()), 0.0)
    dS = P * (do1 @ v1[first].T - D)
    soft, hard = dS.abs() + P * E, P * (do1.abs() @ v1[first].abs().T + D.abs() + E)
    ref = P.T @ do1
    tol = (2.0**-8 + 2.0**-11) * P.T @ do1.abs() + 2.0**-8 * ref.abs()
    near(grads[2][first, 0], ref.cpu().numpy(), tol.cpu().numpy(), "dv")
    ref = scale * dS.T @ q1
    tol = scale * (2.0**-8 * soft + 2.0**-11 * hard).T @ q1.abs() + 2.0**-8 * ref.abs()
    near(grads[1][first, 0], ref.cpu().numpy(), tol.cpu().numpy(), "dk")
    assert all(bool(torch.isfinite(x.float().sum())) for x in grads)


@pytest.mark.parametrize("d,T,ramp", [(16, 2_400_000, None), (128, 2_400_000, None), (64, 500_000, (0.1, 3.0)),
                                      (64, 500_000, (3.0, 0.1)), (128, 400_000, (0.1, 2.0)),
                                      (128, 400_000, (2.0, 0.1))])
def test_window_forward_of_long_sums(d, T, ramp):
    """Rows that see up to 2.4 million keys. With values of one sign the accumulators of the tensor core
    alone lose 1.4 % of them; with a ramp the largest scores come late or early."""
    g = torch.Generator(device=dev()).manual_seed(12)
    T += 130                                                # a short user before the long one
    q, k, v = (torch.randn(T, 1, d, generator=g, device=dev()) for _ in range(3))
    if ramp is None:
        v = v.abs()
    else:
        k *= torch.linspace(*ramp, T, device=dev())[:, None, None]
    q, k, v = (x.to(torch.bfloat16) for x in (q, k, v))
    off, st = torch.tensor([0, 130, T], device=dev()), jca.new_status(dev())
    out, lse = torch.full_like(q, float("nan")), torch.full((T, 1), float("nan"), device=dev())
    jca.jagged_window_attn_fwd(q, k, v, out, off, 1 << 40, 0, lse=lse, status=st)
    jca.check_status(st)
    assert bool(torch.isfinite(out.float().sum()))
    j = torch.arange(T, device=dev())
    for rows in (torch.arange(T - 20, T, device=dev()), torch.arange(T // 2, T // 2 + 20, device=dev()),
                 torch.tensor([130, 131, 131_000, 131_500, 262_400], device=dev())):
        S = d**-0.5 * q[rows, 0].double() @ k[:, 0].double().T
        S.masked_fill_((j[None] > rows[:, None]) | (j[None] < 130), -float("inf"))
        want = torch.logsumexp(S, 1)
        P = torch.exp(S - want[:, None])
        ref, A = P @ v[:, 0].double(), P @ v[:, 0].double().abs()
        # The file's tolerance, and 2^13 additions cut at 2^-23 of the sum.
        tol = (2.0**-8 + 2.0**-11 + 2.0**-10) * A + 2.0**-8 * ref.abs()
        near(out[rows, 0], ref.cpu().numpy(), tol.cpu().numpy(), "out")
        assert float((lse[rows, 0].double() - want).abs().max()) <= 2.0**-11


@pytest.mark.parametrize("d,window,sinks", [(16, 400_000, 3), (64, 300_000, 0), (128, 350_000, 70)])
def test_window_long_rows_with_padding(d, window, sinks):
    """Long sums together with what else a row may have: padding (not finite), first tokens behind a window
    that is long itself, shared heads, short users around. Rows and keys sampled at the ends of tiles."""
    n, H = 500_000, 2
    off_np = np.array([0, 200, 200 + n, 200 + n + 77])
    T, s, e = int(off_np[-1]), 200, 200 + n
    g = torch.Generator(device=dev()).manual_seed(13)
    x = torch.randn(T, H + 2, d, generator=g, device=dev()).to(torch.bfloat16)
    do = torch.randn(T, H, d, generator=g, device=dev()).to(torch.bfloat16)
    valid = (torch.rand(T, generator=g, device=dev()) > 0.1).to(torch.uint8)
    valid[s:s + 2], valid[e - 1], valid[0] = 0, 1, 1
    x[valid == 0], do[valid == 0] = float("nan"), float("inf")
    q, k, v = x.split([H, 1, 1], 1)
    off, st = torch.tensor(off_np, device=dev()), jca.new_status(dev())
    out, lse = torch.full((T, H, d), float("nan"), dtype=torch.bfloat16, device=dev()), torch.empty(T, H, device=dev())
    jca.jagged_window_attn_fwd(q, k, v, out, off, window, sinks, valid=valid, lse=lse, status=st)
    grads = [torch.full((T, h, d), float("nan"), dtype=torch.bfloat16, device=dev()) for h in (H, 1, 1)]
    jca.jagged_window_attn_bwd(q, k, v, out, do, lse, *grads, off, window, sinks, valid=valid, status=st)
    jca.check_status(st)
    real = valid.bool()
    for y in [out] + grads:
        assert bool(torch.isfinite(y.float().sum())) and bool((y[~real] == 0).all())
    clean = torch.where(real[:, None, None], x, 0).double()
    kk, vv = clean[:, H], clean[:, H + 1]
    dd = torch.where(real[:, None, None], do, 0).double()
    scale, j = d**-0.5, torch.arange(T, device=dev())
    rows = torch.tensor([s + 2, s + window - 1, s + window + 1, e - 130, e - 1], device=dev())
    rows = rows[real[rows]]
    seen = real[None] & (j[None] >= s) & (j[None] <= rows[:, None])
    seen &= (j[None] > rows[:, None] - window) | (j[None] < s + sinks)
    keys = torch.tensor([s + 2, s + 3, s + 128, s + 70, e - window, e - 1], device=dev())
    keys = keys[real[keys]]
    sees = real[:, None] & (j[:, None] < e) & (j[:, None] >= keys[None])
    sees &= (j[:, None] - window < keys[None]) | (keys[None] < s + sinks)
    dk, dv, tk, tv = 0, 0, 0, 0
    for h in range(H):
        qq, o1, d1 = clean[:, h], out[:, h].double(), dd[:, h]
        D, E = (d1 * o1).sum(1, keepdim=True), (d1 * o1).abs().sum(1, keepdim=True)
        S = (scale * qq[rows] @ kk.T).masked_fill(~seen, -float("inf"))
        want = torch.logsumexp(S, 1)
        assert float((lse[rows, h].double() - want).abs().max()) <= 2.0**-11
        P = torch.exp(S - want[:, None])
        ref, A = P @ vv, P @ vv.abs()
        near(out[rows, h], ref.cpu().numpy(), ((2.0**-8 + 2.0**-11) * A + 2.0**-8 * ref.abs()).cpu().numpy(), "out")
        dS = P * (d1[rows] @ vv.T - D[rows])
        soft, hard = dS.abs() + P * E[rows], P * (d1[rows].abs() @ vv.abs().T + D[rows].abs() + E[rows])
        ref = scale * dS @ kk
        tol = scale * (2.0**-8 * soft + 2.0**-11 * hard) @ kk.abs() + 2.0**-8 * ref.abs()
        near(grads[0][rows, h], ref.cpu().numpy(), tol.cpu().numpy(), "dq")
        P = torch.where(sees, torch.exp(scale * qq @ kk[keys].T - torch.where(real, lse[:, h].double(), 0)[:, None]), 0.0)
        dS = P * (d1 @ vv[keys].T - D)
        soft, hard = dS.abs() + P * E, P * (d1.abs() @ vv[keys].abs().T + D.abs() + E)
        dk, dv = dk + scale * dS.T @ qq, dv + P.T @ d1
        tk = tk + scale * (2.0**-8 * soft + 2.0**-11 * hard).T @ qq.abs()
        tv = tv + (2.0**-8 + 2.0**-11) * P.T @ d1.abs()
    near(grads[1][keys, 0], dk.cpu().numpy(), (tk + 2.0**-8 * dk.abs()).cpu().numpy(), "dk")
    near(grads[2][keys, 0], dv.cpu().numpy(), (tv + 2.0**-8 * dv.abs()).cpu().numpy(), "dv")


@pytest.mark.parametrize("op", ["rope", "fwd", "bwd", "decode", "tree"])
def test_many_users_of_few_rows(op):
    """1.3 million users, nearly all of them without a row: more than blocks of a grid dimension."""
    rng = np.random.default_rng(4)
    B = 1_300_000
    lens = (rng.random(B) < 0.003) * rng.integers(1, 30, B)
    off_np = np.concatenate([[0], np.cumsum(lens)])
    T = int(off_np[-1])
    g = torch.Generator(device=dev()).manual_seed(5)
    q, k, v = (torch.randn(T, h, 16, generator=g, device=dev()).to(torch.bfloat16) for h in (2, 1, 1))
    off, st, out = torch.tensor(off_np, device=dev()), jca.new_status(dev()), torch.full_like(q, float("nan"))
    some = np.flatnonzero(lens)[rng.integers(0, (lens > 0).sum(), 40)]
    runs = [(slice(int(off_np[u]), int(off_np[u + 1])), int(lens[u])) for u in some]
    if op == "rope":
        pos = torch.arange(T, device=dev())
        jca.jca_rope_axes_fwd(q, None, out, None, pos, [8])
        _rope_check(q.cpu(), out, pos.cpu().numpy()[:, None], [8], False, 1.0, op)
        return
    if op in ("fwd", "bwd"):
        lse, grads = torch.empty(T, 2, device=dev()), [torch.full_like(x, float("nan")) for x in (q, k, v)]
        jca.jagged_window_attn_fwd(q, k, v, out, off, 9, 2, lse=lse, status=st)
        jca.jagged_window_attn_bwd(q, k, v, out, q, lse, *grads, off, 9, 2, status=st)
        jca.check_status(st)
        for r, n in runs:
            mask = lh.window_mask(n, 9, 2)
            ref, _, _, A = lh.masked(q[r], k[r], v[r], mask, 0.25)
            near(out[r], ref, (2.0**-8 + 2.0**-11) * A + 2.0**-8 * np.abs(ref), op)
            ref, tol = lh.gradients(q[r], k[r], v[r], q[r], mask, 0.25)
            for got, x, (soft, hard) in zip(grads, ref, tol):
                near(got[r], x, 2.0**-8 * soft + 2.0**-11 * hard + 2.0**-8 * np.abs(x) + 1e-30, op)
        return
    if op == "tree":
        parent = torch.full((T,), -1, dtype=torch.int32, device=dev())
        jca.cand_tree_attn_fwd(q, k, v, off, parent, v, k, off, out, 29, status=st)
        jca.check_status(st)
        for r, n in runs:
            ref, _, _, A = lh.masked(q[r], torch.cat([v[r], k[r]]), torch.cat([k[r], v[r]]), lh.tree_mask([-1] * n, n), 0.25)
            near(out[r], ref, (2.0**-8 + 2.0**-11) * A + 2.0**-8 * np.abs(ref), op)
        return
    coff = np.concatenate([[0], np.cumsum(lens + 1)])
    kc, vc = (torch.randn(int(coff[-1]), 1, 16, generator=g, device=dev()).to(torch.bfloat16) for _ in range(2))
    q, kn, vn = (torch.randn(B, h, 16, generator=g, device=dev()).to(torch.bfloat16) for h in (2, 1, 1))
    out = torch.full_like(q, float("nan"))
    jca.jagged_window_decode_fwd(q, kn, vn, kc, vc, out, torch.tensor(coff, device=dev()),
                                 torch.tensor(lens, device=dev()), 9, 2, status=st)
    jca.check_status(st)
    for u in [0, B - 1] + list(some):
        r, n = slice(int(coff[u]), int(coff[u + 1])), int(lens[u]) + 1
        ref, _, _, A = lh.masked(q[u:u + 1], kc[r], vc[r], lh.window_mask(n, 9, 2)[-1:], 0.25)
        near(out[u:u + 1], ref, (2.0**-8 + 2.0**-11) * A + 2.0**-8 * np.abs(ref), op)
    assert torch.equal(kc[torch.tensor(coff[1:] - 1, device=dev())], kn)
