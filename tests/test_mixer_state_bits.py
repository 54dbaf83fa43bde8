"""How many bits computed values keep on the way to a prompt's state (qdr_prompt).

S, R = v - decay S^T k, T = (I + L)^-1 diag(beta), U = T R and the decayed U
enter their products as three bfloat16 parts, 24 bits: an fp32 value.  Two parts
would be 16 bits, which a bound on a whole prompt's error hardly tells apart:
here the values are such that what the third part holds adds up.

x = 1 + 2^-9 + 2^-17 - 2^-20 is 1 + 2^-9 in two parts; what is left, 7/8 2^-17 =
112 u (u = 2^-24), is the same everywhere.  One token's k is 1/2 in four
channels (norm 1), so K S has four products that are not 0, of equal sign; every
other token's k is 0.

"carried": S_0 = x, v = 0, beta = x / 2, gate 1.  K S = 2 x errs by 4 u 2 x (four
sums), R by u 2 x, U = -x^2 by 13 u (6 u in the sums of its six products of
parts, 2 u in the three that are left out, 5 u from R), k U by half of that, and
S = x - x^2 / 2 by 3 u more: 10 u.
"decayed": SUM, S_0 = 0, v = 1, gate g = x / 2 at the next token:
S = k g.  log2 g (near -1) errs by 2 u, which is 1.4 u of g, 2^ by 2 u of it, the
sum of its parts, the smallest first, by u: 5 u of g / 2.
"map": as "carried" in a prompt of several segments, the token in the second:
its map is I - (x / 2) k k^T, whose entries err by 4 u (13 u / 2 of U = x / 4, and
a sum's u), and the join adds four of them times x (16 u), in sums that err by 10 u: 30 u.
Every bound is asserted for a plain model of the arithmetic here, which also
shows that it fails when one operand has two parts.
"""
import numpy as np
import pytest

from quantized_delta_rule_decode_amd import qdr

D, U = 128, 2.0 ** -24
X = np.float32(1 + 2.0 ** -9 + 2.0 ** -17 - 2.0 ** -20)
Y = X / np.float32(2)
CHANNELS = [3, 40, 77, 126]
ROOM = {"carried": 10 * U, "decayed": 1.25 * U, "map": 30 * U}
OPERANDS = {"carried": ["S", "R", "T", "U"], "decayed": ["U"], "map": ["S", "P"]}


def expected(name):
    """A state's entry in the four channels (fp64), and in the others."""
    x, y = float(X), float(Y)
    return (y / 2, 0.0) if name == "decayed" else (x - y * x, x)


def part(x):
    """fp32 to nearest-even bfloat16."""
    w = np.asarray(x, np.float32).view(np.uint32)
    return ((w + np.uint32(0x7FFF) + ((w >> np.uint32(16)) & np.uint32(1))) & np.uint32(0xFFFF0000)).view(np.float32)


def cut(x, parts):
    out, left = np.float32(0), np.float32(x)
    for _ in range(parts):
        p = part(left)
        out, left = np.float32(out + p), np.float32(left - p)
    return out


def model(name, two=None):
    """The entry in the four channels, in fp32, with operand `two` in two parts."""
    f = np.float32
    keep = lambda x, operand: cut(x, 2 if operand == two else 3)    # noqa: E731
    half = f(0.5)
    if name == "decayed":
        return half * keep(f(np.exp2(f(np.log2(Y)))), "U")
    if name == "map":
        # P's row of one of the channels, then P S
        u = -f(Y * half)
        own, other = keep(f(f(1) + half * u), "P"), keep(half * u, "P")
        s = keep(X, "S")
        total = f(own * s)
        for _ in range(3):
            total = f(total + f(other * s))
        return total
    ks = f(0)
    for _ in CHANNELS:
        ks = f(ks + half * keep(X, "S"))
    u = f(keep(Y, "T") * keep(f(-ks), "R"))
    return f(X + half * keep(u, "U"))


@pytest.mark.parametrize("name", list(ROOM))
def test_the_bounds_tell_two_parts_from_three(name):
    want = expected(name)[0]
    assert abs(float(model(name)) - want) <= ROOM[name]
    for operand in OPERANDS[name]:
        off = abs(float(model(name, operand)) - want)
        assert off > ROOM[name] * 1.5, f"{operand} in two parts is off by {off / U:.1f} u, the bound is {ROOM[name] / U:.1f} u"


# heads, tokens: four workgroups a head; one; several segments
CASES = [("carried", 2, 1), ("carried", 2, 200), ("carried", 130, 70), ("decayed", 2, 70), ("decayed", 2, 1500), ("decayed", 600, 70), ("map", 2, 2300)]


@pytest.mark.gpu
@pytest.mark.parametrize("name,H,T", CASES)
def test_state_keeps_three_parts(name, H, T):
    import torch
    qdr.load()
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")       # noqa: E731
    at = {"carried": T // 2, "decayed": 5, "map": 300}[name]
    carried = name != "decayed"
    q, k, v = (torch.zeros((T, H, D), dtype=torch.bfloat16, device="cuda") for _ in range(3))
    k[at, :, CHANNELS] = 0.5
    beta, gate = torch.full((T, H), float(Y), device="cuda"), torch.ones((T, H), device="cuda")
    if not carried:
        v[at] = 1
        gate[at + 1] = float(Y)
    with qdr.Pool(1, H, [qdr.K_FP32] * H, None, scale_mode=qdr.SCALE_ROW_ABSMAX) as pool:
        pool.qdr_pack(i32([0]), torch.full((1, H, D, D), float(X), device="cuda"))
        pool.qdr_prompt(qdr.RULE_DELTA if carried else qdr.RULE_SUM, i32([0]), i32([0, T]), q, k, v, beta if carried else None, gate,
                        torch.empty_like(q), carry=i32([1]) if carried else None)
        S = torch.empty((1, H, D, D), device="cuda")
        pool.qdr_unpack(i32([0]), S)
    S = S[0].double().cpu().numpy()
    inside, outside = expected(name)
    off = np.abs(S[:, CHANNELS] - inside).max()
    assert off <= ROOM[name], f"off by {off / U:.1f} u, the bound is {ROOM[name] / U:.1f} u"
    others = np.ones(D, bool)
    others[CHANNELS] = False
    assert (S[:, others] == outside).all()
