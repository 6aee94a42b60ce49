"""The serving calls at the largest sizes that they take."""
import pytest
import torch

import verifiable_quantize_rows_gb300 as bsg

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("N", [65535 * 512, 65535 * 512 + 1, (1 << 25) - 1, 1 << 25])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
def test_products_of_the_most_columns(N, dtype):
    """Each column's bits are those of a call on a few columns (65 rows of K are two units in one split)."""
    K, M = 65, 5
    g = torch.Generator("cuda").manual_seed(1)
    Q, sc = bsg.wquant_groups(torch.randn((K, N), generator=g, device="cuda"), 32)
    X = torch.randn((M, K), generator=g, device="cuda").to(dtype)
    Y = bsg.wgroups_matvec(X, Q, sc, group=32)
    for c in (0, 512 * 40000, 512 * 65534, N // 512 * 512 - 512):
        part = slice(c, min(N, c + 1024))
        q = Q[:, c // 2:(part.stop + 1) // 2]
        assert torch.equal(Y[:, part], bsg.wgroups_matvec(X, q, sc[:, part], group=32))


@pytest.mark.parametrize("T,heads", [(16, 40000), (1, 65535)])
def test_attention_of_the_most_heads(T, heads):
    """Each head's bits are those of a call on a few heads (one page: one chunk)."""
    D, page, length = 256 if T > 1 else 32, 16, 16
    g = torch.Generator("cuda").manual_seed(1)
    codes = [torch.randint(-127, 128, (1, heads, page, D), generator=g, device="cuda").to(torch.int8) for _ in range(2)]
    scales = [torch.rand((1, heads), generator=g, device="cuda") + 0.1 for _ in range(2)]
    q = torch.randn((1, T, heads, D), generator=g, device="cuda") * 0.01
    table, lens = torch.zeros((1, 1), dtype=torch.int32, device="cuda"), torch.full((1,), length, dtype=torch.int32, device="cuda")
    o = bsg.kv8_attend(q, bsg.Kv8Cache(*codes, *scales), table, lens)
    for h in (0, heads // 2, 32760, heads - 8):
        few = slice(h, h + 8)
        cache = bsg.Kv8Cache(*[c[:, few].contiguous() for c in (*codes, *scales)])
        assert torch.equal(o[:, :, few], bsg.kv8_attend(q[:, :, few], cache, table, lens))


def test_more_rows_than_a_call_takes():
    """The refusal names no other call: none takes codes with group scales."""
    Q, sc = bsg.wquant_groups(torch.randn((64, 40), device="cuda"), 32)
    with pytest.raises(ValueError, match=r"at most 16 rows a call: X has 17$"):
        bsg.wgroups_matvec(torch.ones((17, 64), device="cuda"), Q, sc, group=32)


def test_rows_that_overlap_are_refused_by_name():
    Q, sc = bsg.wquant_groups(torch.randn((64, 40), device="cuda"), 32)
    x, row = torch.ones((3, 64), device="cuda"), torch.ones((1, 64), device="cuda").expand(3, 64)
    close = torch.ones(200, device="cuda").as_strided((3, 64), (63, 1))
    lse, out = torch.zeros(3, device="cuda"), torch.empty((1, 40), device="cuda").expand(3, 40)
    for name, call in (("W", lambda: bsg.wquant_groups(row)), ("X", lambda: bsg.wgroups_matvec(row, Q, sc, group=32)),
                       ("X", lambda: bsg.wgroups_matvec(close, Q, sc, group=32)),
                       ("Q", lambda: bsg.wgroups_matvec(x, Q[:1].expand(64, 20), sc, group=32)),
                       ("scale", lambda: bsg.wgroups_matvec(x, Q, sc[:1].expand(2, 40), group=32)),
                       ("out", lambda: bsg.wgroups_matvec(x, Q, sc, group=32, out=out)),
                       ("logits", lambda: bsg.logprobs(row)), ("logits", lambda: bsg.logprobs_backward(row, None, lse)),
                       ("out", lambda: bsg.logprobs_backward(x, None, lse, out=row))):
        with pytest.raises(ValueError, match=f"the rows of {name} must not overlap"):
            call()


def test_products_do_not_go_where_their_rows_are():
    Q, sc = bsg.wquant_groups(torch.randn((64, 64), device="cuda"), 32)
    x = torch.ones((2, 64), device="cuda")
    with pytest.raises(ValueError, match="out must not share X's memory"):
        bsg.wgroups_matvec(x, Q, sc, group=32, out=x)
    assert (x == 1).all()
