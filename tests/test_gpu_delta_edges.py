"""Calls of the gated delta rule and of the queries' and keys' norms that their
documentation allows at its edges: strides beyond 32 bits, broadcast inputs,
values that are not finite, the smallest numbers of a type, borders of lanes
and workgroups, two threads on two streams, given outputs."""
import threading

import pytest

torch = pytest.importorskip("torch")

import delta_reference as R  # noqa: E402
from test_gpu_delta import DT, check_delta, check_norm, fields, generator  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def fm():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import fft_block_toeplitz_amd as fm

    fm.lib()
    return fm


def apart(tensors, batch, step):
    """Copies of [batch, steps, ...] tensors in one memory, rows `step` and sequences `batch` elements apart, one tensor
    behind the other in each row."""
    widths = [t[0, 0].numel() for t in tensors]
    B, T = tensors[0].shape[:2]
    base = torch.empty((B - 1) * batch + (T - 1) * step + sum(widths), dtype=tensors[0].dtype, device="cuda")
    out, at = [], 0
    for t, w in zip(tensors, widths):
        inner = t[0, 0].stride()
        view = base.as_strided(t.shape, (batch, step, *inner), at)
        view.copy_(t)
        out.append(view)
        at += w
    return out


@pytest.mark.parametrize("batch,step,T", [(2 ** 31 + 8, 512, 70), (2 ** 31 + 7, 511, 70), (1, 2 ** 24, 140)])
def test_far_apart(fm, batch, step, T):
    """Sequences and steps whose distance does not fit in 32 bits: what contiguous copies give."""
    B = 2 if batch > 1 else 1
    x = [t.contiguous() for t in fields(1, (B, T), 2, 4, 32, 16, "bf16")]
    far = apart(x, batch, step)
    dy = torch.randn((B, T, 4, 16), generator=generator(2), device="cuda").bfloat16()
    y, last, carries = fm.delta_rule(*x, save=True)
    y2, last2, carries2 = fm.delta_rule(*far, save=True)
    tol = R.tolerance(torch.bfloat16)
    R.near(y2, y.double(), 2 * tol, "y", rows=False)
    R.near(last2, last.double(), 128 * R.U, "last states", rows=False)
    grads, far_grads = fm.delta_rule_backward(dy, *x, carries), fm.delta_rule_backward(dy, *far, carries2)
    for name, a, b in zip("dq dk dv dgate dbeta dh0".split(), far_grads, grads):
        # two results that are each `tol` off in the norm; dgate sums what cancels, a few times its own size
        R.near(a, b.double(), (8 if name == "dgate" else 2) * tol, name, rows=False)
    w = torch.ones(32, device="cuda")
    for a, b in zip(fm.qk_norm(far[0], far[1], w, w), fm.qk_norm(x[0], x[1], w, w)):
        assert torch.equal(a, b)
    for a, b in zip(fm.qk_norm_backward(far[0], far[1], far[0], far[1], w, w),
                    fm.qk_norm_backward(x[0], x[1], x[0], x[1], w, w)):
        assert torch.equal(a, b)


def test_far_places(fm):
    """A cache whose places are more than 2^31 elements apart."""
    x = [t[:, 0] for t in fields(3, (2, 1), 1, 2, 16, 24, "fp32")]
    near = torch.randn((2, 2, 16, 24), generator=generator(4), device="cuda")
    far = torch.empty(2 ** 31 + 2 ** 10, device="cuda").as_strided(near.shape, (2 ** 31 + 8, *near.stride()[1:]))
    far.copy_(near)
    slots = torch.tensor([1, 0], dtype=torch.int32, device="cuda")
    assert torch.equal(fm.delta_rule_step(*x, far, slots), fm.delta_rule_step(*x, near, slots))
    assert torch.equal(far, near)


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
def test_broadcast_inputs(fm, dtype):
    """Inputs expanded over sequences, steps and heads, and the gradients that autograd sums for them."""
    gen, dt = generator(5), DT[dtype]
    n = lambda *s: torch.randn(s, generator=gen, device="cuda").to(dt)  # noqa: E731
    q, k = (torch.nn.functional.normalize(n(1, 100, 1, 24).float(), dim=-1).to(dt) for _ in range(2))
    small = [q, k, n(2, 1, 1, 16), n(1, 1, 3), n(2, 100, 1)]
    shapes = [(2, 100, 3, 24), (2, 100, 3, 24), (2, 100, 3, 16), (2, 100, 3), (2, 100, 3)]
    dy, dl = n(2, 100, 3, 16), torch.randn((2, 3, 24, 16), generator=gen, device="cuda")

    def run(leaves, widen):
        y, last = fm.delta_rule(*(widen(t.expand(s)) for t, s in zip(leaves, shapes)))
        return y, last, *torch.autograd.grad((y, last), leaves, (dy, dl))

    got = run([t.clone().requires_grad_() for t in small], lambda t: t)
    want = run([t.clone().requires_grad_() for t in small], lambda t: t.contiguous())
    tol = R.tolerance(dt)
    for i, (a, b) in enumerate(zip(got, want)):
        R.near(a, b.double(), (8 if i == 5 else 2) * tol, f"output {i}", rows=False)
    q = small[0].expand(2, 100, 3, 24)
    for a, b in zip(fm.qk_norm(q, q), fm.qk_norm(q.contiguous(), q.contiguous())):
        assert torch.equal(a, b)


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
@pytest.mark.parametrize("dtype,V", [("fp32", 24), ("bf16", 72)])
def test_not_finite_stays_where_it_is(fm, bad, dtype, V):
    """One value that is not finite: other sequences and other heads keep their bits, and so do the runs in front of it."""
    x = fields(6, (3, 200), 2, 4, 32, V, dtype)
    dy = torch.randn((3, 200, 4, V), generator=generator(7), device="cuda").to(DT[dtype])
    y, last, carries = fm.delta_rule(*x, save=True)
    grads = fm.delta_rule_backward(dy, *x, carries)
    x[2][1, 130, 3, 5] = bad
    y2, last2, carries2 = fm.delta_rule(*x, save=True)
    grads2 = fm.delta_rule_backward(dy, *x, carries2)
    assert not torch.isfinite(y2[1, 130, 3]).all() and not torch.isfinite(last2[1, 3]).all()
    assert torch.equal(y2[1, :128, 3], y[1, :128, 3])
    for a, b in ((y2, y), (grads2[2], grads[2]), (grads2[3], grads[3]), (grads2[4], grads[4])):
        assert torch.equal(a[[0, 2]], b[[0, 2]]) and torch.equal(a[1, :, :3], b[1, :, :3])
    for a, b in ((last2, last), (grads2[5], grads[5])):
        assert torch.equal(a[[0, 2]], b[[0, 2]]) and torch.equal(a[1, :3], b[1, :3])
    for a, b in zip(grads2[:2], grads[:2]):  # heads 2 and 3 share the queries and keys of head 1
        assert torch.equal(a[[0, 2]], b[[0, 2]]) and torch.equal(a[1, :, 0], b[1, :, 0])
    q = x[0].clone()
    q[1, 7, 0, 3] = bad
    w = torch.ones(32, device="cuda")
    (a, c), (b, d) = fm.qk_norm(q, x[1], w, w), fm.qk_norm(x[0], x[1], w, w)
    assert not torch.isfinite(a[1, 7, 0]).all()
    a[1, 7, 0] = b[1, 7, 0]
    assert torch.equal(a, b) and torch.equal(c, d)


def test_delta_small_halves(fm):
    """FP16 keys and queries of which a part are subnormal numbers: all of their bits take part."""
    def change(q, k, v, gate, beta):
        q *= 2.0 ** -13
        k[..., 8:] *= 2.0 ** -14
        v[..., :2] *= 2.0 ** -14

    # y is taken where its values are large enough for the type, the states, in 32 bits, everywhere
    x = fields(8, (1, 150), 1, 2, 24, 20, "fp16")
    change(*x)
    want = R.delta_rule(*(t[0].double() for t in x), torch.zeros((2, 24, 20), dtype=torch.float64, device="cuda"),
                        "sigmoid", "sigmoid", 2.0 ** 13)
    y, last = fm.delta_rule(*x, scale=2.0 ** 13)
    for h in range(2):
        R.near(last[0, h], want[1][h], 64 * R.U, "last states", rows=False)
        R.near(last[0, h, 8:], want[1][h, 8:], 64 * R.U, "last states under small keys", rows=False)
        R.near(y[0, :, h, 2:], want[0][:, h, 2:], R.tolerance(torch.float16), "y", rows=False)


@pytest.mark.parametrize("D,n", [(8, 4), (9, 4), (9, 0), (7, 0), (10, 3), (16, 3), (16, 4), (23, 7), (65, 32), (66, 29),
                                 (511, 253), (512, 253), (505, 250), (510, 255), (33, 9), (264, 100)])
@pytest.mark.parametrize("pairs", ["halves", "neighbours"])
def test_qk_norm_borders_of_lanes(fm, D, n, pairs):
    """Parts of heads that end inside a lane, are shorter than one, or take all lanes and one more."""
    check_norm(fm, D + n, (2, 21), 3, 2, D, "fp32", "rms", pairs, n, True)
    check_norm(fm, D - n, (1, 19), 5, 1, D, "bf16", "l2", pairs, n, True, strided=True)


@pytest.mark.parametrize("rows,Hq,Hk", [((4000,), 1, 1), ((3, 700), 70, 1), ((2, 513), 1, 300), ((1, 5000), 7, 3)])
def test_qk_norm_many_rows(fm, rows, Hq, Hk):
    """More rows than the workgroups of a backward call take at once, and heads that are no multiple of a workgroup's."""
    lengths = None if len(rows) == 1 else [rows[1] - 100] * rows[0]
    check_norm(fm, Hq, rows, Hq, Hk, 40, "fp16", "rms", "halves", 10, True, lengths=lengths)


def test_two_threads_on_two_streams(fm):
    """The same calls from two threads at once, each on its own stream."""
    sets = [fields(20 + i, (2, 300), 2, 2, 64, 64, "bf16") for i in range(2)]
    dy = torch.randn((2, 300, 2, 64), generator=generator(9), device="cuda").bfloat16()
    w = torch.ones(64, device="cuda")

    def work(x):
        q, k = fm.qk_norm(x[0], x[1], w, w, norm="l2")
        y, last, carries = fm.delta_rule(q, k, *x[2:], save=True)
        grads = fm.delta_rule_backward(dy, q, k, *x[2:], carries)
        return y, last, *grads, *fm.qk_norm_backward(grads[0], grads[1], x[0], x[1], w, w, norm="l2")

    want = [work(x) for x in sets]
    torch.cuda.synchronize()
    got, errors = [None, None], []

    def thread(i):
        try:
            stream = torch.cuda.Stream()
            with torch.cuda.stream(stream):
                for _ in range(20):
                    got[i] = work(sets[i])
            stream.synchronize()
        except Exception as e:  # noqa: BLE001
            errors.append(e)

    threads = [threading.Thread(target=thread, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors, errors
    for a, b in zip(got, want):
        assert all(torch.equal(s, t) for s, t in zip(a, b))


def test_given_outputs(fm):
    x = fields(10, (2, 70), 1, 2, 16, 24, "bf16")
    out = torch.full_like(x[2], float("nan"))
    y, last = fm.delta_rule(*x, out=out)
    assert y is out and torch.equal(out, fm.delta_rule(*x)[0])
    one = [t[:, 0] for t in x]
    state = torch.randn((3, 2, 16, 24), generator=generator(11), device="cuda")
    again, out = state.clone(), torch.full((2, 2, 24), float("nan"), device="cuda", dtype=torch.bfloat16)
    slots = torch.tensor([2, 5], dtype=torch.int32, device="cuda")
    assert fm.delta_rule_step(*one, state, slots, out=out) is out
    assert torch.equal(out, fm.delta_rule_step(*one, again, slots)) and torch.equal(state, again) and not out[1].any()


def test_queries_and_keys_of_one_memory(fm):
    """Queries that are the keys, and values beside them: inputs may overlap."""
    def change(q, k, v, gate, beta):
        q.copy_(k)

    check_delta(fm, 12, 2, 130, 1, 2, 32, 32, "fp32", change=change)
    x = fields(13, (1, 90), 1, 1, 32, 32, "bf16")
    same = fm.delta_rule(x[1], x[1], x[1], *x[3:])
    copies = fm.delta_rule(x[1].clone(), x[1].clone(), x[1].clone(), *x[3:])
    assert torch.equal(same[0], copies[0]) and torch.equal(same[1], copies[1])


@pytest.mark.parametrize("B,packed", [(130, False), (129, True), (600, False), (530, True)])
def test_many_ragged_sequences(fm, B, packed):
    """More chains than run at once, lengths of all kinds: each sequence as in a call of a few, whatever its place."""
    gen = generator(B)
    lengths = torch.randint(0, 200, (B,), generator=gen, device="cuda", dtype=torch.int32)
    lengths[:4] = torch.tensor([0, 200, 1, 64], dtype=torch.int32)
    lengths[7] = lengths[8]
    x = fields(14, (B, 200), 1, 2, 16, 72, "bf16")
    dy = torch.randn((B, 200, 2, 72), generator=gen, device="cuda").bfloat16()
    h0, dl = (torch.randn((B, 2, 16, 72), generator=gen, device="cuda") for _ in range(2))
    hold = torch.arange(200, device="cuda")[None] < lengths[:, None]

    def run(pick):
        n = lengths[pick].contiguous()
        if packed:
            how = {"offsets": torch.cat([n[:1] * 0, n.cumsum(0).to(torch.int32)])}
            a = [t[pick][hold[pick]] for t in (*x, dy)]
        else:
            how, a = {"lengths": n}, [t[pick].contiguous() for t in (*x, dy)]
        y, last, carries = fm.delta_rule(*a[:5], h0[pick].contiguous(), save=True, **how)
        *grads, dh0 = fm.delta_rule_backward(a[5], *a[:5], carries, h0[pick].contiguous(), dl[pick].contiguous(), **how)
        rows = [y, *grads] if packed else [t[hold[pick]] for t in (y, *grads)]
        ends = n.cumsum(0).tolist()
        return [[t[e - int(m):e] for e, m in zip(ends, n)] for t in rows] + [list(last), list(dh0)]

    everything = run(torch.arange(B, device="cuda"))
    backwards = run(torch.arange(B - 1, -1, -1, device="cuda"))
    few = run(torch.arange(9, device="cuda"))
    for a, b, c in zip(everything, backwards, few):
        assert all(torch.equal(s, t) for s, t in zip(a, reversed(b)))
        assert all(torch.equal(s, t) for s, t in zip(a[:9], c))
