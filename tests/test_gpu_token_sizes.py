"""The token path on the GPU on both sides of the sizes at which its kernels change
their way: tables and outputs beyond the L2 cache, borders of the sort's shares and
of the sums' pieces, heads read two at a time, float32 rows into the cache."""
import pytest
import torch

import test_gpu_embed as embed
import test_gpu_qk_rope as qk
from test_gpu_paged_attn import Batch

pytestmark = pytest.mark.gpu
BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32


# ---------------------------------------------------------------- embedding

TABLES = [
    # tokens, h, vocab, dtype, scale: tables above 48 MB, whose last rows are filled beside the sums
    (700, 1024, 30011, BF16, 1.5),
    (1, 8192, 4000, BF16, 1.0),  # one piece
    (5000, 2056, 7001, F32, 1.0),  # runs over many pieces, ragged column tiles
    (300, 136, 200003, F16, 3.0),
    (900, 13, 2000003, BF16, 1.0),  # single elements
    (64, 40960, 700, BF16, 1.0),  # a row at a time
]


@pytest.mark.parametrize("how", ["any", "last", "outside"])
@pytest.mark.parametrize("case", TABLES, ids=lambda c: f"{c[0]}x{c[1]}-of-{c[2]}-{str(c[3])[6:]}")
def test_gradient_of_a_large_table_is_written_whole(cuda_lib, case, how):
    """|error| ≤ eps/2·|ref| + (n + 2)·2^-24·scale·Σ|dx| as for the small tables; every row is written, nothing
    behind the table."""
    M, h, vocab, dt, scale = case
    assert vocab * h * dt.itemsize > 48 << 20
    g = torch.Generator(device="cuda").manual_seed(M)
    tok = torch.randint(0, vocab, (M,), generator=g, device="cuda")
    if how == "last":  # the rows on both sides of the first filled one, and the table's last
        first = (48 << 20) // (h * dt.itemsize)
        rows = torch.tensor([0, first - 1, first, first + 1, vocab - 2, vocab - 1], device="cuda")
        tok = rows[torch.randint(0, len(rows), (M,), generator=g, device="cuda")]
    if how == "outside":
        tok = torch.where(torch.rand(M, generator=g, device="cuda") < 0.5, tok, -1)
    dx = torch.randn(M, 1, h, generator=g, device="cuda").to(dt)
    buf = torch.full((vocab * h + 64,), float("nan"), dtype=dt, device="cuda")
    buf[vocab * h :] = 7.5
    got = buf[: vocab * h].view(vocab, h)
    cuda_lib.embed_backward(tok.view(M, 1), dx, got, s=M, b=1, h=h, vocab=vocab, tp=1, scale=scale)
    assert (buf[vocab * h :] == 7.5).all()
    ok = (tok >= 0).nonzero().view(-1)
    rows, at = torch.unique(tok[ok], return_inverse=True)
    sums = torch.zeros(3, len(rows), h, dtype=torch.float64, device="cuda")
    for j, part in enumerate((dx[ok, 0].double() * scale, dx[ok, 0].double().abs() * scale, torch.ones_like(dx[ok, 0]).double())):
        sums[j].index_add_(0, at, part)
    ref, size, count = sums
    tol = torch.finfo(dt).eps / 2 * ref.abs() + (count + 2) * 2.0**-24 * size + 2.0**-25 * (dt == F16)
    assert ((got[rows].double() - ref).abs() <= tol).all()
    untouched = torch.ones(vocab, dtype=torch.bool, device="cuda")
    untouched[rows] = False
    assert not got[untouched].any()


@pytest.mark.parametrize("mb", [63, 111, 112, 130])
@pytest.mark.parametrize("dt,h,tp", [(BF16, 8192, 8), (F16, 1000, 1), (F32, 4100, 2)])
def test_large_lookups_are_the_rounded_product(cuda_lib, dt, h, tp, mb):
    """Outputs that L2 keeps, that nearly fill it and that pass through it."""
    vocab, scale = 3001, 1.7
    s = (mb << 20) // (h * dt.itemsize) // tp * tp + (0 if mb == 111 else tp)
    g = torch.Generator(device="cuda").manual_seed(mb)
    tok = torch.randint(-1, vocab + 1, (s, 1), generator=g, device="cuda")
    table = torch.randn(vocab, h, generator=g, device="cuda").to(dt)
    out = [torch.full((s // tp, 1, h), float("nan"), dtype=dt, device="cuda") for _ in range(tp)]
    cuda_lib.embed_forward(tok, table, out, s=s, b=1, h=h, vocab=vocab, tp=tp, scale=scale)
    ok = (tok >= 0) & (tok < vocab)
    product = (table.float() * torch.tensor(scale, device="cuda")).to(dt)
    want = torch.where(ok[..., None], product[tok.clamp(0, vocab - 1)], torch.zeros((), dtype=dt, device="cuda"))
    assert torch.equal(torch.cat(out), want)


BORDERS = [512, 513,  # tokens that one CTA sorts
           32768, 32769,  # 128 tokens a warp stay in registers
           14576, 14577, 29152, 29153, 58304, 58305]  # pieces of 8, 16, 32 and 64 rows


@pytest.mark.parametrize("main_grad", [False, True], ids=["table", "main_grad"])
@pytest.mark.parametrize("s", BORDERS)
def test_gradient_at_the_borders_of_sort_and_pieces(cuda_lib, s, main_grad):
    embed.test_gradient_against_the_oracle(cuda_lib, (s, 1, 16, 611, 1, BF16, "out", True, 1.3), main_grad)


# ---------------------------------------------------------------- QK norm and rotation

ROWS32 = [
    # rows, b, heads, kv, d, rot, interleaved, norm, dtype, positions
    (40, 2, 8, 2, 128, 128, True, True, F32, True),
    (30, 1, 6, 3, 64, 32, False, True, F32, False),
    (11, 1, 5, 5, 80, 80, False, False, F32, False),
    (12, 1, 16, 2, 256, 16, False, True, F32, False),
    (900, 1, 32, 8, 128, 128, False, True, F32, True),  # several heads a lane group
]
ROWS32_IDS = [f"m{c[0]}-{c[2]}x{c[3]}x{c[4]}" for c in ROWS32]


@pytest.mark.parametrize("case", ROWS32, ids=ROWS32_IDS)
def test_float32_rows(cuda_lib, case):
    qk.test_forward(cuda_lib, case)
    qk.test_backward(cuda_lib, case)


@pytest.mark.parametrize("layout", ["page-token-head", "page-head-token"])
@pytest.mark.parametrize("case", ROWS32, ids=ROWS32_IDS)
def test_float32_rows_into_the_cache(cuda_lib, case, layout):
    qk.test_append(cuda_lib, case, layout)


# ---------------------------------------------------------------- paged attention

PAIRS = [
    # lengths, heads, kv heads, page, dtype: heads of 96 side by side in a page
    ([300, 17, 0, 1], 64, 64, 16, BF16),
    ([2900, 1200, 31, 32, 33], 24, 8, 32, F16),
    ([700, 1], 12, 4, 7, BF16),  # pages that end inside a tile
    ([130, 0, 2000], 40, 2, 16, F16),  # 20 heads a group: two blocks
    ([65, 900], 32, 1, 16, BF16),  # the two units are blocks of one group
    ([90, 511, 3], 6, 3, 16, BF16),  # an odd number of units: one at a time
    ([20000], 4, 2, 64, BF16),  # one pair of units over every CTA
    ([40] * 50, 16, 16, 16, F16),
]


@pytest.mark.parametrize("case", PAIRS, ids=[f"{len(c[0])}x{max(c[0])}-{c[1]}x{c[2]}-p{c[3]}-{str(c[4])[6:]}" for c in PAIRS])
def test_neighbouring_heads_of_96(cuda_lib, case):
    lengths, heads, kv, page, dt = case
    x = Batch(lengths, heads, kv, 96, page, dt)
    o, lse = x.run(cuda_lib)
    assert cuda_lib.device_status() == 0, cuda_lib.last_error()
    x.check(o, lse)
