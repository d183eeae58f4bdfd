"""Long caches in which every 64 keys count: for tests that must see a single unit of keys lost,
doubled or taken from elsewhere, which random inputs do not show (their outputs shrink with the
number of keys, and any of them has next to no weight).

Each query head of a KV head's group has a query of its own, the same for all tokens.  Every
unit of 64 keys holds one key along the query of one head of the group (the units in turn),
whose score of about 14 leaves all other keys less than a thousandth of the weight.  Its value
is 1 in one dimension, its neighbours' in others, so that an output element is the share of the
c planted keys that have it.  Losing or doubling one of them changes that element by 1/c of its
value or more; the error bound allows 2^-8 for the weights, 2^-8 for the result and 2^-10 for
the scores, 1/110."""
import torch

SCORE = 14.0
UNIT = 64
PLACES = (0, 63, 15, 16, 31, 32, 47, 48)   # of the planted key within its unit


def queries(gen, T, Hq, d, device):
    """q [T, Hq, d], the same row for every token."""
    return torch.randn(Hq, d, generator=gen).to(torch.bfloat16).to(device).expand(T, Hq, d).clone()


def plant(q, k, v):
    """Plants the keys and values of a sequence, q [T, Hq, d], k, v [S, Hkv, d], in place; returns
    each planted key's place [n], head within the group [n] and dimension [n]."""
    Hq, d = q.shape[1:]
    S, Hkv = k.shape[:2]
    G = Hq // Hkv
    unit = torch.arange(-(-S // UNIT), device=k.device)
    head, turn = unit % G, unit // G
    at = UNIT * unit + torch.tensor(PLACES, device=k.device)[turn % len(PLACES)]
    at = at.clamp(max=S - 1)
    dim = (41 * turn) % d
    for g in range(Hkv):
        u = q[0, g * G:(g + 1) * G].double()
        u = SCORE * u / u.norm(dim=1, keepdim=True) * d ** 0.5 / u.norm(dim=1, keepdim=True)
        k[at, g] = u[head].to(k.dtype)
        v[at, g] = torch.nn.functional.one_hot(dim, d).to(v.dtype)
    return at, head, dim
