"""The prompt form of the recurrences (qdr_prompt) and the additive step
(qdr_linear_step) against the recurrence itself, token by token in 64 bits:

    S_t = a_t S_{t-1} + k_t u_t^T,  o_t = S_t^T q_t,
    u_t = v_t (SUM) or beta_t (v_t - a_t S_{t-1}^T k_t) (DELTA).

Tolerances.  u = 2^-24 is the fp32 half step.  A chunk's sums have up to 384
products (128 or 64 terms in up to three bfloat16 parts) and the triangular
solve amplifies by a small factor; the transitions (I - beta k k^T) a are no
larger than 1 in norm, so one chunk's error is not amplified by the later
ones: |S - ref|_F <= 1024 u (chunks + 1) max_t |S_t|_F (the measured error is
some 2^-24).  The readout of chunk row t sums m = 2^g |q|^T |S_0| + sum |A||u|
in operands of two bfloat16 parts (2^-16 each, three of them) and is then
rounded to bfloat16 (2^-8 of the value):
|o - ref| <= 2^-8 |ref| + 4 2^-16 m + the state's error times |q|.
The step's sums are fp32: |S - ref| <= 3 u (|a S| + |k v|), and its readout
<= 130 u sum |q||S| (+ 2^-8 |ref| with bfloat16 outputs).
"""
import numpy as np
import pytest

from quantized_delta_rule_decode_amd import qdr

pytestmark = pytest.mark.gpu
D, C = 128, 64
U = 2.0 ** -24
DELTA, SUM = qdr.RULE_DELTA, qdr.RULE_SUM


@pytest.fixture(scope="module")
def torch_dev():
    import torch
    assert torch.cuda.is_available(), "device tests need a HIP GPU"
    qdr.load()
    return torch


def fp32_pool(n, H):
    return qdr.Pool(n, H, [qdr.K_FP32] * H, None, scale_mode=qdr.SCALE_ROW_ABSMAX)


def i32(torch, x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def make(torch, seed, T, H, gates="mixed"):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    rn = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
    unit = lambda x: x / x.norm(dim=-1, keepdim=True)           # noqa: E731
    u = torch.rand((T, H), generator=g, device="cuda")
    gate = {"mixed": torch.exp2(-torch.exp2(-10 * u)), "one": torch.ones_like(u), "small": u ** 4,
            "zeros": torch.where(u < 0.2, 0.0, u), "tiny": torch.full_like(u, 1e-30)}[gates]
    return dict(q=(unit(rn(T, H, D)) / D ** 0.5).bfloat16(), k=unit(rn(T, H, D)).bfloat16(), v=rn(T, H, D).bfloat16(),
                beta=torch.rand((T, H), generator=g, device="cuda"), gate=gate.contiguous())


def reference(torch, x, rule, S, first, length):
    """One sequence in fp64: o, m (see above), the last state, and the largest norm of any state, a head."""
    H = x["q"].shape[1]
    q, k, v, beta, gate = (x[n][first:first + length].double() for n in ("q", "k", "v", "beta", "gate"))
    o, m = torch.zeros((length, H, D), dtype=torch.float64, device="cuda"), torch.zeros((length, H, D), dtype=torch.float64, device="cuda")
    most = S.flatten(1).norm(dim=1)
    for t in range(length):
        if t % C == 0:
            start, us, ks, dec, head = S.clone(), [], [], [], torch.ones(H, dtype=torch.float64, device="cuda")
        a = gate[t]
        S = a[:, None, None] * S
        u = v[t] if rule == SUM else beta[t][:, None] * (v[t] - (k[t][:, None, :] @ S)[:, 0])
        S = S + k[t][:, :, None] * u[:, None, :]
        most = torch.maximum(most, S.flatten(1).norm(dim=1))
        o[t] = (q[t][:, None, :] @ S)[:, 0]
        head, dec = head * a, [d * a for d in dec] + [torch.ones_like(a)]
        us.append(u), ks.append(k[t])
        m[t] = head[:, None] * (q[t].abs()[:, None, :] @ start.abs())[:, 0]
        for d, kk, uu in zip(dec, ks, us):
            m[t] += (d * (q[t] * kk).sum(-1).abs())[:, None] * uu.abs()
    return o, m, S, most


def run(torch, pool, rule, slots, lens, x, carry=None, lead=0, tail=0, **kw):
    """o (rows outside the sequences hold 7) of one call."""
    T, H = x["q"].shape[0], x["q"].shape[1]
    cu = i32(torch, np.concatenate([[lead], lead + np.cumsum(lens)]).tolist())
    assert lead + sum(lens) + tail == T
    o = torch.full((T, H, D), 7.0, dtype=torch.bfloat16, device="cuda")
    pool.qdr_prompt(rule, i32(torch, slots), cu, x["q"], x["k"], x["v"], x["beta"] if rule == DELTA else None, x["gate"], o,
                    carry=None if carry is None else i32(torch, carry), **kw)
    return o


def states(torch, pool, slots):
    S = torch.empty((len(slots), pool.num_heads, D, D), device="cuda")
    pool.qdr_unpack(i32(torch, slots), S)
    return S


def check(torch, x, rule, lens, lead, o, S, S0):
    at = lead
    for b, n in enumerate(lens):
        ref, m, last, most = reference(torch, x, rule, S0[b].double(), at, n)
        slack = 1024 * U * (-(-n // C) + 1) * most
        err = (S[b].double() - last).flatten(1).norm(dim=1)
        assert (err <= slack).all(), f"sequence {b}: state off by {err.tolist()} of {most.tolist()}"
        room = 2.0 ** -8 * ref.abs() + 4 * 2.0 ** -16 * m + (slack * x["q"][at:at + n].double().norm(dim=-1))[..., None]
        off = (o[at:at + n].double() - ref).abs()
        assert (off <= room).all(), f"sequence {b}: readout off by {(off - room).max().item():.3g} over its bound"
        at += n


LENGTHS = [[1], [63], [64], [65], [0, 5, 130, 1, 64], [200, 3]]


@pytest.mark.parametrize("rule", [DELTA, SUM])
@pytest.mark.parametrize("lens", LENGTHS, ids=str)
@pytest.mark.parametrize("carried", [False, True])
def test_prompt_against_the_recurrence(torch_dev, rule, lens, carried):
    torch = torch_dev
    n, H, lead, tail = len(lens), 3, 2, 5
    x = make(torch, 11 + sum(lens), lead + sum(lens) + tail, H)
    pool = fp32_pool(n + 2, H)
    slots = [(b + 1) % (n + 2) for b in range(n)][::-1]
    S0 = torch.randn((n, H, D, D), device="cuda", generator=torch.Generator(device="cuda").manual_seed(3))
    pool.qdr_pack(i32(torch, slots), S0)
    carry = [b % 3 != 1 for b in range(n)] if carried else None
    o = run(torch, pool, rule, slots, lens, x, carry, lead, tail)
    assert (o[:lead] == 7).all() and (o[lead + sum(lens):] == 7).all(), "rows outside the sequences were written"
    keep = torch.tensor([bool(carried and c) for c in (carry or [0] * n)], device="cuda")
    check(torch, x, rule, lens, lead, o, states(torch, pool, slots), S0 * keep[:, None, None, None])
    assert pool.qdr_poll_device_error() == 0


@pytest.mark.parametrize("rule", [DELTA, SUM])
@pytest.mark.parametrize("gates", ["one", "small", "zeros", "tiny"])
def test_prompt_gates(torch_dev, rule, gates):
    torch = torch_dev
    lens, H = [150, 40], 2
    x = make(torch, 5, sum(lens), H, gates)
    if rule == DELTA:
        x["beta"][10:20] = 0
        x["beta"][20:30] = 1
    pool = fp32_pool(2, H)
    S0 = torch.randn((2, H, D, D), device="cuda", generator=torch.Generator(device="cuda").manual_seed(4))
    pool.qdr_pack(i32(torch, [0, 1]), S0)
    o = run(torch, pool, rule, [0, 1], lens, x, [1, 1])
    check(torch, x, rule, lens, 0, o, states(torch, pool, [0, 1]), S0)


@pytest.mark.parametrize("rule", [DELTA, SUM])
def test_prompt_many_heads(torch_dev, rule):
    """Enough (sequence, head) pairs for the launch that takes wider slices."""
    torch = torch_dev
    lens, H = [70, 1, 90, 0, 65, 129], 33
    x = make(torch, 6, sum(lens), H)
    pool = fp32_pool(6, H)
    S0 = torch.randn((6, H, D, D), device="cuda", generator=torch.Generator(device="cuda").manual_seed(2))
    slots, carry = [3, 1, 0, 5, 2, 4], [1, 0, 0, 1, 1, 0]
    pool.qdr_pack(i32(torch, slots), S0)
    o = run(torch, pool, rule, slots, lens, x, carry)
    check(torch, x, rule, lens, 0, o, states(torch, pool, slots), S0 * torch.tensor(carry, device="cuda")[:, None, None, None])
    pool.qdr_slot_reset(i32(torch, slots))
    p = run(torch, pool, rule, [3, 1, -1, 5, 2, 9], lens, x)
    assert torch.equal(p[71 + 90:71 + 90 + 65], run(torch, pool, rule, [0, 1, 2, 3, 4, 5], lens, x)[71 + 90:71 + 90 + 65])
    assert (p[71:161] == 0).all() and (p[226:] == 0).all()
    assert pool.qdr_poll_device_error() == qdr.DEVERR_SLOT


@pytest.mark.parametrize("lens,carried,gates", [([2200], True, "one"), ([2500, 0, 1500], False, "mixed"), ([1344, 1656], True, "zeros")], ids=str)
def test_long_delta_prompts(torch_dev, lens, carried, gates):
    """Prompts of several segments, joined by their maps of states."""
    torch = torch_dev
    n, H = len(lens), 2
    x = make(torch, 17, sum(lens), H, gates)
    pool = fp32_pool(n, H)
    slots = list(range(n))[::-1]
    S0 = torch.randn((n, H, D, D), device="cuda", generator=torch.Generator(device="cuda").manual_seed(3))
    pool.qdr_pack(i32(torch, slots), S0)
    o = run(torch, pool, DELTA, slots, lens, x, [1] * n if carried else None)
    check(torch, x, DELTA, lens, 0, o, states(torch, pool, slots), S0 * float(carried))
    # some are padding, and the first is the only one that continues
    pool.qdr_pack(i32(torch, slots), S0)
    p = run(torch, pool, DELTA, slots[:1] + [-1] * (n - 1), lens, x, [1] + [0] * (n - 1))
    assert not p[lens[0]:].any()
    first = {k: y[:lens[0]].contiguous() for k, y in x.items()}
    check(torch, first, DELTA, lens[:1], 0, p[:lens[0]], states(torch, pool, slots[:1]), S0[:1])
    assert torch.equal(states(torch, pool, slots[1:]), S0[1:])
    packed = qdr.Pool(n, H, [8, 16], np.ones((H, D), np.float32))
    packed.qdr_pack(i32(torch, slots), S0)
    start = states(torch, packed, slots)
    o = run(torch, packed, DELTA, slots, lens, x, [1] * n if carried else None)
    dense = fp32_pool(n, H)
    dense.qdr_pack(i32(torch, slots), start)
    assert torch.equal(o, run(torch, dense, DELTA, slots, lens, x, [1] * n if carried else None))


@pytest.mark.parametrize("packed", [False, True], ids=["uncompressed", "quantised"])
def test_long_delta_prompts_hand_on_the_state_they_continue(torch_dev, packed):
    """The first segment's readout starts from the workspace, as the others'
    do: the last segment's workgroup writes the slot in the same launch.  So
    the state a prompt continues from stands there when the call is done."""
    torch = torch_dev
    lens, H = [2500, 40, 1460], 2
    x = make(torch, 18, sum(lens), H)
    pool = qdr.Pool(3, H, [8, 16], np.ones((H, D), np.float32)) if packed else fp32_pool(3, H)
    slots, carry = [2, 0, 1], [1, 1, 0]
    S0 = torch.randn((3, H, D, D), device="cuda", generator=torch.Generator(device="cuda").manual_seed(6))
    pool.qdr_pack(i32(torch, slots), S0)
    S0 = states(torch, pool, slots)
    ws = torch.zeros(pool.qdr_prompt_workspace(3, sum(lens)), dtype=torch.uint8, device="cuda")
    o = run(torch, pool, DELTA, slots, lens, x, carry, workspace=ws)
    held = torch.isin(S0[0].view(torch.int32), ws.view(torch.int32))
    assert held.all(), f"{(~held).sum().item()} of {held.numel()} values of the state are not handed on"
    dense = fp32_pool(3, H)
    dense.qdr_pack(i32(torch, slots), S0)
    assert torch.equal(o, run(torch, dense, DELTA, slots, lens, x, carry))
    check(torch, x, DELTA, lens, 0, o, states(torch, dense, slots), S0 * torch.tensor(carry, device="cuda")[:, None, None, None])


def test_prompt_non_finite_in_segments(torch_dev):
    """Values that are not finite in one head of a long prompt."""
    torch = torch_dev
    H, T = 3, 2300
    pool = fp32_pool(1, H)
    x = make(torch, 19, T, H)
    for rule in (DELTA, SUM):
        ref = run(torch, pool, rule, [0], [T], x)
        for name, value in (("k", float("nan")), ("v", float("inf")), ("gate", float("nan"))):
            y = {m: t.clone() for m, t in x.items()}
            y[name][700, 1] = value
            o = run(torch, pool, rule, [0], [T], y)
            assert torch.equal(o[:640], ref[:640]) and torch.equal(o[:, [0, 2]], ref[:, [0, 2]])
            # (an infinite value times one score is an infinity, summed with others of its column NaN)
            assert (~o[700:, 1].isfinite()).any(dim=-1).all(), (rule, name)
            S = states(torch, pool, [0])[0].isfinite()
            assert not S[1].all() and S[[0, 2]].all()
    pool.close()


@pytest.mark.parametrize("lens,carried", [([1200], True), ([700, 0, 257, 64, 1], False), ([256, 512, 300], True)], ids=str)
def test_long_additive_prompts(torch_dev, lens, carried):
    """Prompts of several segments, with padding and gates that forget."""
    torch = torch_dev
    n, H = len(lens), 2
    x = make(torch, 16, sum(lens), H, "zeros" if carried else "mixed")
    pool = fp32_pool(n, H)
    slots = list(range(n))[::-1]
    S0 = torch.randn((n, H, D, D), device="cuda", generator=torch.Generator(device="cuda").manual_seed(3))
    pool.qdr_pack(i32(torch, slots), S0)
    o = run(torch, pool, SUM, slots, lens, x, [1] * n if carried else None)
    check(torch, x, SUM, lens, 0, o, states(torch, pool, slots), S0 * float(carried))
    packed = qdr.Pool(n, H, [8, 16], np.ones((H, D), np.float32))
    packed.qdr_pack(i32(torch, slots), S0)
    start = states(torch, packed, slots)
    o = run(torch, packed, SUM, slots[:1] + [-1] * (n - 1), lens, x, [1] * n if carried else None)
    assert (o[lens[0]:] == 0).all()
    dense = fp32_pool(1, H)
    dense.qdr_pack(i32(torch, [0]), start[:1].contiguous())
    first = {k: y[:lens[0]].contiguous() for k, y in x.items()}
    ref = run(torch, dense, SUM, [0], lens[:1], first, [1] if carried else None)
    check(torch, first, SUM, lens[:1], 0, o[:lens[0]], states(torch, dense, [0]), start[:1] * float(carried))
    check(torch, first, SUM, lens[:1], 0, ref, states(torch, dense, [0]), start[:1] * float(carried))


def test_parts_of_a_prompt_equal_the_whole(torch_dev):
    """A prompt in two calls cut at a chunk's end is the prompt in one, bit for bit."""
    torch = torch_dev
    H = 2
    x = make(torch, 8, 64 + 77, H)
    for rule in (DELTA, SUM):
        one, two = fp32_pool(1, H), fp32_pool(1, H)
        whole = run(torch, one, rule, [0], [141], x)
        part = lambda a, b: {k: y[a:b].contiguous() for k, y in x.items()}  # noqa: E731
        a = run(torch, two, rule, [0], [64], part(0, 64))
        b = run(torch, two, rule, [0], [77], part(64, 141), [1])
        assert torch.equal(torch.cat([a, b]), whole)
        assert np.array_equal(one.qdr_read_raw(0), two.qdr_read_raw(0))


POOLS = {
    "heads": dict(kinds=[8, 16, 6, 4, 32, 2], unit=qdr.UNIT_HEAD),
    "heads_refit_bf16": dict(kinds=[2, 6, 2], unit=qdr.UNIT_HEAD, fit_iters=1, scale_bits=16),
    "rows": dict(kinds=([16] + [8] * 15 + [6] * 32 + [4] * 48 + [2] * 32) * 2, unit=qdr.UNIT_ROW),
}


@pytest.mark.parametrize("name", list(POOLS))
@pytest.mark.parametrize("rule", [DELTA, SUM])
def test_prompt_into_a_quantised_pool(torch_dev, name, rule):
    """The slots hold what qdr_pack stores of the state that an uncompressed
    pool ends with; a carried prompt starts from what qdr_unpack restores."""
    torch = torch_dev
    kw = dict(POOLS[name])
    kinds = np.array(kw.pop("kinds"), np.uint8)
    H = kinds.size if kw["unit"] == qdr.UNIT_HEAD else kinds.size // D
    omega = np.random.default_rng(3).lognormal(0, 1, (H, D)).astype(np.float32)
    new = lambda: qdr.Pool(4, H, kinds, omega, **kw)  # noqa: E731
    dev, twin, dense = new(), new(), fp32_pool(4, H)
    every = i32(torch, [0, 1, 2, 3])
    for p in (dev, twin):
        p.qdr_slot_reset(every)
    slots, lens = [2, 0, -1, 3], [100, 0, 70, 1]
    for turn, carry in enumerate([None, [1, 1, 1, 0], [0, 0, 0, 1]]):
        x = make(torch, 20 + turn, sum(lens), H)
        dense.qdr_pack(every, states(torch, twin, [0, 1, 2, 3]))
        before = [twin.qdr_read_raw(s) for s in range(4)]
        ref = run(torch, dense, rule, slots, lens, x, carry)
        got = run(torch, dev, rule, slots, lens, x, carry)
        assert torch.equal(got, ref)
        assert (got[100:170] == 0).all(), "a padding sequence's rows are 0"
        done = [s for b, s in enumerate(slots) if s >= 0 and not (lens[b] == 0 and carry and carry[b])]
        twin.qdr_pack(i32(torch, done), states(torch, dense, done))
        for s in range(4):
            assert np.array_equal(dev.qdr_read_raw(s), twin.qdr_read_raw(s)), f"turn {turn}: slot {s}"
            if s not in done:
                assert np.array_equal(dev.qdr_read_raw(s), before[s])
    assert dev.qdr_poll_device_error() == 0


def test_prompt_then_steps(torch_dev):
    """Prompt and steps together, as they are used: a prompt into the pool and
    then single tokens equal the whole sequence as one prompt (uncompressed)."""
    torch = torch_dev
    H, n, length = 3, 2, 90
    x = make(torch, 31, n * (length + 3), H)
    rows = lambda b, a, e: slice(b * (length + 3) + a, b * (length + 3) + e)  # noqa: E731
    whole = {r: fp32_pool(n, H) for r in (DELTA, SUM)}
    o_ref = {r: run(torch, whole[r], r, [0, 1], [length + 3] * n, x) for r in whole}
    head = {k: torch.cat([y[rows(b, 0, length)] for b in range(n)]) for k, y in x.items()}
    for rule in (DELTA, SUM):
        pool = fp32_pool(n, H)
        run(torch, pool, rule, [0, 1], [length] * n, head)
        for t in range(length, length + 3):
            q, k, v, beta, gate = (torch.stack([x[m][rows(b, t, t + 1)][0] for b in range(n)]) for m in ("q", "k", "v", "beta", "gate"))
            o = torch.empty_like(q)
            if rule == DELTA:
                pool.qdr_decode_step_bf16(i32(torch, [0, 1]), q, k, v, beta, gate, o)
            else:
                pool.qdr_linear_step_bf16(i32(torch, [0, 1]), q, k, v, gate, o)
            for b in range(n):
                ref = o_ref[rule][rows(b, t, t + 1)][0].double()
                # two roundings to bfloat16, and |q| times the states' difference
                assert ((o[b].double() - ref).abs() <= 2 * 2.0 ** -8 * ref.abs() + 2.0 ** -12).all()
        A, B = states(torch, pool, [0, 1]).double(), states(torch, whole[rule], [0, 1]).double()
        assert (A - B).norm() <= 1024 * U * 3 * B.norm()


def test_prompt_non_finite_stays_in_its_head(torch_dev):
    torch = torch_dev
    lens, H = [130, 130], 3
    x = make(torch, 41, 260, H)
    ref = run(torch, fp32_pool(2, H), DELTA, [0, 1], lens, x)
    for name, bad in (("v", float("nan")), ("k", float("inf")), ("gate", float("nan")), ("gate", -0.5), ("beta", float("inf"))):
        y = {k: t.clone() for k, t in x.items()}
        y[name][100, 1] = bad                        # sequence 0, second chunk, head 1
        pool = fp32_pool(2, H)
        o = run(torch, pool, DELTA, [0, 1], lens, y)
        assert torch.equal(o[:64], ref[:64]) and torch.equal(o[130:], ref[130:])
        assert torch.equal(o[:, [0, 2]], ref[:, [0, 2]])
        assert o[100:130, 1].isnan().any(dim=-1).all(), name
        assert states(torch, pool, [0])[0, 1].isnan().any()
        pool.close()


def test_prompt_errors_on_the_device(torch_dev):
    torch = torch_dev
    H = 2
    x = make(torch, 51, 100, H)
    pool = fp32_pool(2, H)
    pool.qdr_slot_reset(i32(torch, [0, 1]))
    o = run(torch, pool, DELTA, [5, 0], [40, 60], x)
    assert (o[:40] == 0).all() and pool.qdr_poll_device_error() == qdr.DEVERR_SLOT
    # counts that leave the rows, or go back
    for cu in ([0, 40, 101], [0, 60, 40], [-1, 40, 100], [0, 2 ** 31 - 1, 100]):
        o = torch.full((100, H, D), 7.0, dtype=torch.bfloat16, device="cuda")
        pool.qdr_prompt(DELTA, i32(torch, [0, 1]), i32(torch, cu), x["q"], x["k"], x["v"], x["beta"], x["gate"], o)
        assert pool.qdr_poll_device_error() == qdr.DEVERR_LENGTH, cu
    # and where sequences are cut into segments
    T = 4000
    x = make(torch, 52, T, H)
    for cu in ([0, T, 5, T], [0, T + 1, T + 1, T + 1], [0, 400, 400, 2 ** 31 - 1], [0, -7, 300, T], [T, 0, 0, 0], [0, 300, 700, 699],
               [0, 2000, 1900, T], [0, 5, T, 3000]):
        for rule in (SUM, DELTA):
            o = torch.full((T, H, D), 7.0, dtype=torch.bfloat16, device="cuda")
            pool.qdr_prompt(rule, i32(torch, [0, -1, 1]), i32(torch, cu), x["q"], x["k"], x["v"], x["beta"], x["gate"], o)
            assert pool.qdr_poll_device_error() == qdr.DEVERR_LENGTH, cu
    pool.close()


@pytest.mark.parametrize("rule", [DELTA, SUM])
@pytest.mark.parametrize("cu", [[0, 512, 256, 4000], [0, 256, 0, 4000], [0, 4000, 3999, 4000]], ids=str)
def test_counts_that_decrease_between_segments(torch_dev, rule, cu):
    """A decreasing pair is told of also where no segment falls to its sequence."""
    torch = torch_dev
    H, T = 2, 4000
    pool, x = fp32_pool(3, H), make(torch, 54, T, H)
    o = torch.full((T, H, D), 7.0, dtype=torch.bfloat16, device="cuda")
    pool.qdr_prompt(rule, i32(torch, [0, 1, 2]), i32(torch, cu), x["q"], x["k"], x["v"], x["beta"], x["gate"], o)
    assert pool.qdr_poll_device_error() == qdr.DEVERR_LENGTH
    pool.close()


@pytest.mark.parametrize("rule", [DELTA, SUM])
def test_prompt_rows_beyond_32_bits(torch_dev, rule):
    """Rows whose elements and bytes are numbered above 2^31 and 2^32."""
    torch = torch_dev
    H, far, L = 64, 262_200, 300
    pool = fp32_pool(2, H)
    y = make(torch, 53, L, H)
    x = {m: torch.empty((far + L, *t.shape[1:]), dtype=t.dtype, device="cuda") for m, t in y.items()}
    for m in y:
        x[m][far:] = y[m]
    o = torch.full((far + L, H, D), 7.0, dtype=torch.bfloat16, device="cuda")
    # the sequence before it is skipped: its rows of o are cleared
    pool.qdr_prompt(rule, i32(torch, [-1, 1]), i32(torch, [0, far, far + L]), x["q"], x["k"], x["v"], x["beta"], x["gate"], o)
    check(torch, y, rule, [L], 0, o[far:], states(torch, pool, [1]), torch.zeros((1, H, D, D), device="cuda"))
    assert not o[:far].any() and pool.qdr_poll_device_error() == 0
    pool.close()


def test_prompt_refusals(torch_dev, monkeypatch):
    torch = torch_dev
    H, T = 2, 10
    x = make(torch, 61, T, H)
    pool = fp32_pool(2, H)
    cu, slots, o = i32(torch, [0, T]), i32(torch, [0]), torch.full((T, H, D), 7.0, dtype=torch.bfloat16, device="cuda")
    args = lambda **k: {**dict(rule=DELTA, slots=slots, cu=cu, o=o, **x), **k}  # noqa: E731
    odd = torch.empty(T * H * D + 1, dtype=torch.bfloat16, device="cuda")[1:].view(T, H, D)
    small = torch.empty(pool.qdr_prompt_workspace(1, T) - 1, dtype=torch.uint8, device="cuda")
    for bad, kind in ((dict(rule=7), qdr.QdrError), (dict(beta=None), qdr.QdrError), (dict(q=odd), qdr.QdrError),
                      (dict(workspace=small), qdr.QdrError), (dict(q=x["q"].float()), TypeError), (dict(q=x["q"][:5]), ValueError),
                      (dict(v=x["v"].transpose(0, 1)), ValueError), (dict(gate=x["gate"][:, :1]), ValueError),
                      (dict(cu=cu.long()), TypeError), (dict(slots=i32(torch, [0, 1])), ValueError), (dict(o=o.cpu()), TypeError)):
        with pytest.raises(kind):
            pool.qdr_prompt(**args(**bad))
    diag = qdr.Pool(2, H, [8] * H, np.ones((H, D), np.float32), gate=qdr.GATE_DIAG)
    with pytest.raises(qdr.QdrError) as ei:
        diag.qdr_prompt(**args())
    assert ei.value.status == -5
    packed = qdr.Pool(2, H, [8] * H, np.ones((H, D), np.float32))
    with pytest.raises(qdr.QdrError) as ei:
        packed.qdr_linear_step(slots, *(x[m][:1].float() for m in "qkv"), x["gate"][:1], o[:1].float())
    assert ei.value.status == -5
    monkeypatch.setenv("QDR_DEBUG", "1")
    with pytest.raises(qdr.QdrError) as ei:
        pool.qdr_prompt(**args(slots=i32(torch, [0, 0]), cu=i32(torch, [0, 4, T])))
    assert ei.value.status == -4
    pool.qdr_prompt(**args(slots=i32(torch, [-1])))       # padding passes the check
    torch.cuda.synchronize()
    assert (o == 0).all()


@pytest.mark.parametrize("rule", [DELTA, SUM])
def test_long_prompts_in_graphs(torch_dev, rule):
    """A prompt that is cut into segments, captured and replayed between eager
    work on the same pool: every replay equals the eager call."""
    torch = torch_dev
    H, lens = 2, [2100, 900]
    T = sum(lens)
    pool, eager = fp32_pool(2, H), fp32_pool(2, H)
    x, slots, cu, carry = make(torch, 91, T, H), i32(torch, [1, 0]), i32(torch, [0, lens[0], T]), i32(torch, [1, 1])
    o, g = torch.zeros((T, H, D), dtype=torch.bfloat16, device="cuda"), torch.cuda.CUDAGraph()
    ws = torch.empty(pool.qdr_prompt_workspace(2, T), dtype=torch.uint8, device="cuda")
    for p in (pool, eager):
        p.qdr_slot_reset(slots)
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        pool.qdr_prompt(rule, slots, cu, x["q"], x["k"], x["v"], x["beta"], x["gate"], o, carry=carry, workspace=ws)
    for turn in range(3):
        for m, t in make(torch, 92 + turn, T, H).items():
            x[m].copy_(t)
        g.replay()
        ref = run(torch, eager, rule, [1, 0], lens, x, [1, 1])
        assert torch.equal(o, ref), turn
        assert torch.equal(states(torch, pool, [0, 1]), states(torch, eager, [0, 1]))
        o.zero_()
    del g


def test_prompt_without_sequences_or_rows(torch_dev):
    torch = torch_dev
    pool = fp32_pool(1, 2)
    pool.qdr_pack(i32(torch, [0]), torch.ones((1, 2, D, D), device="cuda"))
    x = make(torch, 1, 0, 2)
    run(torch, pool, SUM, [], [], x)
    run(torch, pool, SUM, [0], [0], x, [1])
    assert (states(torch, pool, [0]) == 1).all()
    run(torch, pool, SUM, [0], [0], x)
    assert (states(torch, pool, [0]) == 0).all()


def test_prompt_graphs_and_streams(torch_dev):
    """Two captured graphs with workspaces of their own, replayed with eager
    work between, and a call on a side stream: all equal the eager call."""
    torch = torch_dev
    kinds, H, lens = np.array([8, 16, 6], np.uint8), 3, [70, 20]
    omega = np.ones((H, D), np.float32)
    eager, pools = qdr.Pool(2, H, kinds, omega), [qdr.Pool(2, H, kinds, omega) for _ in range(2)]
    x = make(torch, 71, 90, H)
    static = {k: t.clone() for k, t in x.items()}
    slots, cu, carry = i32(torch, [1, 0]), i32(torch, [0, 70, 90]), i32(torch, [1, 0])
    outs, graphs, spaces = [], [], []
    for p in [eager] + pools:
        p.qdr_slot_reset(i32(torch, [0, 1]))
    for p in pools:
        o, g = torch.zeros((90, H, D), dtype=torch.bfloat16, device="cuda"), torch.cuda.CUDAGraph()
        ws = torch.empty(p.qdr_prompt_workspace(2, 90), dtype=torch.uint8, device="cuda")
        torch.cuda.synchronize()
        with torch.cuda.graph(g):
            p.qdr_prompt(DELTA, slots, cu, static["q"], static["k"], static["v"], static["beta"], static["gate"], o, carry=carry, workspace=ws)
        outs.append(o), graphs.append(g), spaces.append(ws)
    for turn in range(4):
        y = make(torch, 80 + turn, 90, H)
        for k, t in y.items():
            static[k].copy_(t)
        torch.cuda.synchronize()
        side = [torch.cuda.Stream() for _ in range(2)]
        for s, g in zip(side, graphs):
            with torch.cuda.stream(s):
                g.replay()
        ref = run(torch, eager, DELTA, [1, 0], lens, y, [1, 0])
        torch.cuda.synchronize()
        for o, p in zip(outs, pools):
            assert torch.equal(o, ref)
            for s in range(2):
                assert np.array_equal(p.qdr_read_raw(s), eager.qdr_read_raw(s))
            o.zero_()
    s = torch.cuda.Stream()
    twin = qdr.Pool(2, H, kinds, omega)
    twin.qdr_slot_reset(i32(torch, [0, 1]))
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        o = run(torch, twin, DELTA, [1, 0], lens, y)
        copy = o.clone()
    s.synchronize()
    assert torch.equal(copy, run(torch, eager, DELTA, [1, 0], lens, y))


@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("B,H", [(1, 1), (3, 5), (40, 7)])
def test_linear_step(torch_dev, bf16, B, H):
    torch = torch_dev
    pool = fp32_pool(B + 2, H)
    g = torch.Generator(device="cuda").manual_seed(B)
    S0 = torch.randn((B + 2, H, D, D), generator=g, device="cuda")
    every = list(range(B + 2))
    pool.qdr_pack(i32(torch, every), S0)
    slots = list(reversed(range(1, B + 1)))
    if B > 2:
        slots[1] = -1
    q, k, v = (torch.randn((B, H, D), generator=g, device="cuda") for _ in range(3))
    gate = torch.rand((B, H), generator=g, device="cuda")
    gate[0] = 0
    if bf16:
        q, k, v = q.bfloat16(), k.bfloat16(), v.bfloat16()
    o = torch.full_like(q, 7)
    (pool.qdr_linear_step_bf16 if bf16 else pool.qdr_linear_step)(i32(torch, slots), q, k, v, gate, o)
    S = states(torch, pool, every).double()
    left = set(every) - set(slots)
    for s in left:
        assert torch.equal(S[s], S0[s].double())
    for b, s in enumerate(slots):
        if s < 0:
            assert (o[b] == 0).all()
            continue
        old, add = gate[b].double()[:, None, None] * S0[s].double(), k[b].double()[:, :, None] * v[b].double()[:, None, :]
        assert ((S[s] - (old + add)).abs() <= 3 * U * (old.abs() + add.abs())).all()
        ref, m = (q[b].double()[:, :, None] * S[s]).sum(1), (q[b].double()[:, :, None] * S[s]).abs().sum(1)
        assert ((o[b].double() - ref).abs() <= 130 * U * m + (2.0 ** -8 * ref.abs() if bf16 else 0)).all()
    assert pool.qdr_poll_device_error() == 0
    o.fill_(7)
    (pool.qdr_linear_step_bf16 if bf16 else pool.qdr_linear_step)(i32(torch, [B + 2] + [-1] * (B - 1)), q, k, v, gate, o)
    assert (o == 0).all() and pool.qdr_poll_device_error() == qdr.DEVERR_SLOT
    assert torch.equal(states(torch, pool, every).double(), S)


def test_calls_follow_a_two_stream_step(torch_dev):
    """A prompt and a step queued right behind the two-stream step see its write-back."""
    torch = torch_dev
    H, n = 2, 64
    x = make(torch, 91, n, H)
    pools = [fp32_pool(n, H) for _ in range(2)]
    slots, cu = i32(torch, list(range(n))), i32(torch, list(range(n + 1)))
    f = [x[m].float().contiguous() for m in "qkv"]
    outs = []
    for split, p in zip((False, True), pools):
        p.qdr_slot_reset(slots)
        o = torch.empty((n, H, D), device="cuda")
        if split:
            wb = torch.cuda.Stream()
            wb.wait_stream(torch.cuda.current_stream())
            p.qdr_decode_step_split(slots, *f, x["beta"], x["gate"], o, torch.cuda.current_stream(), wb)
        else:
            p.qdr_decode_step(slots, *f, x["beta"], x["gate"], o)
        a, b = torch.empty_like(x["q"]), torch.empty_like(o)
        p.qdr_prompt(DELTA, slots, cu, x["q"], x["k"], x["v"], x["beta"], x["gate"], a, carry=torch.ones_like(slots))
        p.qdr_linear_step(slots, *f, x["gate"], b)
        outs.append((a, b))
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(*outs))
