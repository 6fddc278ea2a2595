"""Verification where rows begin off a 16-byte boundary and at the ends of its
arguments' ranges."""
import pytest
import torch

pytestmark = pytest.mark.gpu

S = None


@pytest.fixture(autouse=True)
def _lib():
    global S
    from lossless_kv_cache_bf16_gb300 import splitzip

    S = splitzip


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def greedy(logits, tokens):
    """Chains of [batch, nodes] tokens over logits; path, accepted, next, status."""
    batch, nodes, _ = logits.shape
    parents = torch.arange(-1, nodes - 1, dtype=torch.int32, device="cuda").expand(batch, nodes).contiguous()
    path, accepted, nxt, status = (torch.full(s, -7, dtype=torch.int32, device="cuda") for s in ((batch, nodes), (batch,), (batch,), (1,)))
    S.sz_verify_tree(logits, tokens, parents, 1.0, path, accepted, nxt, status=status)
    return path, accepted, nxt, int(status)


def placed(shape, dtype, off):
    """A tensor whose first element lies `off` elements behind a 16-byte boundary."""
    n = 1
    for s in shape:
        n *= s
    return torch.full((n + 8,), -2.0, dtype=dtype, device="cuda")[off:off + n].view(shape)


@pytest.mark.parametrize("off", range(8))
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("vocab", [3, 9, 64, 4999, 5000, 40001])
def test_equal_logits(vocab, dtype, off):
    """Rows of one value: token 0, and a child with it is accepted."""
    logits = placed((6, 3, vocab), dtype, off)
    tokens = i32([[0, 0, vocab - 1]]).expand(6, 3).contiguous()
    path, accepted, nxt, status = greedy(logits, tokens)
    assert path.tolist() == [[0, 1, -1]] * 6 and accepted.tolist() == [2] * 6 and nxt.tolist() == [0] * 6 and status == 0


@pytest.mark.parametrize("off", range(8))
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("vocab", [120, 121, 5000, 4999])
def test_two_equal_logits(vocab, dtype, off):
    """Every pair of a token among the first and one a little behind, and of one
    among the last and one a little before it: the lower is the next one, the
    higher as a child is not accepted, the lower is."""
    pairs = [(a, z) for a in range(8) for z in range(a + 1, 80)]
    pairs += [(vocab - 1 - z, vocab - 1 - a) for a, z in pairs]
    n = len(pairs)
    low, high = torch.tensor(pairs, device="cuda").T
    logits = placed((n, 2, vocab), dtype, off)
    logits.scatter_(2, low[:, None, None].expand(n, 2, 1), 1.5)
    logits.scatter_(2, high[:, None, None].expand(n, 2, 1), 1.5)
    for child, took in ((high, 1), (low, 2)):
        tokens = torch.stack([torch.zeros_like(child), child], 1).int()
        _, accepted, nxt, status = greedy(logits, tokens)
        assert torch.equal(nxt.long(), low) and bool((accepted == took).all()) and status == 0


@pytest.mark.parametrize("mode", ["certain", "draft", "greedy"])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("scale", [1e30, 1e38, 2.0 ** 127])
def test_lowest_temperatures(scale, dtype, mode):
    """Products of a logit and the scale that fp32 does not hold; their differences
    decide.  The 64-bit walk is good up to scales of 1e10, where ln 2 is still
    seen beside a product.  Differences of these logits are 0 or above 1e-7, so
    that from there on only the largest logits have any weight and every scale
    gives the same."""
    from tests import test_gpu_verify as verify

    verify.S = S
    for vocab in (60, 5003):
        c = verify.Case(20, 5, vocab, "tree", mode, dtype, seed=34)
        c.logits = torch.where(torch.arange(20)[:, None, None] < 10, c.logits, c.logits - 30).to(dtype)
        c.scale = float(torch.tensor(1e10))
        want = c.check()
        assert want[3] == 0 and all(0 <= x < vocab for x in want[2])
        assert c.run(scale=float(torch.tensor(scale))) == want
