"""fa_fwd_score in the form that long prompts run: items of 256 rows, two stages
of 128 that walk the key tiles together, stage 0 joining late or stopping early,
with every modification; whole and with the keys split.  Each shape asserts the
plan that it is here for.  Bounds: ops_ref.py."""
import pytest
import torch

from attention_forward_gb300 import fa
import ops_ref

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "fp16": torch.float16}


@pytest.fixture(scope="module", autouse=True)
def built():
    import __graft_entry__
    __graft_entry__.build()
    assert torch.cuda.is_available()


def make(B, H, Hkv, Sq, Skv, D, dt, seed):
    g = torch.Generator("cuda").manual_seed(seed)
    n = lambda *s: torch.randn(s, generator=g, device="cuda").to(DT[dt])  # noqa: E731
    return n(B, H, Sq, D), n(B, Hkv, Skv, D), n(B, Hkv, Skv, D)


def documents(B, Sq, Skv):
    """Documents of 1 to 150 keys, cuts inside items and stages, the last 3 keys
    in none; the other batch rows' in another order."""
    dk = torch.zeros((B, Skv), dtype=torch.int32)
    at, n = 0, 0
    for d in range(Skv):
        if d - at >= (1, 37, 90, 128, 150, 11, 64)[n % 7]:
            at, n = d, n + 1
        dk[:, d] = n
    dk[:, Skv - 3:] = -1
    dk[1::2] = dk[1::2].flip(1)
    dq = torch.full((B, Sq), -1, dtype=torch.int32)
    m = min(Sq, Skv)
    dq[:, Sq - m:] = dk[:, Skv - m:]
    return dq.cuda(), dk.cuda()


# name: (type, arguments); True stands for an array made for the shape
FORMS = {
    "plain": ("bf16", dict(causal=True)),
    "plain full": ("fp16", dict()),
    "cap": ("bf16", dict(causal=True, softcap=30.0)),
    "cap full": ("bf16", dict(softcap=30.0)),
    "cap running": ("fp16", dict(causal=True, softcap=20.0)),
    "cap 100": ("bf16", dict(causal=True, softcap=100.0)),
    "bias": ("fp16", dict(causal=True, slopes=True)),
    "bias full": ("bf16", dict(slopes=True)),
    "cap bias": ("bf16", dict(causal=True, softcap=30.0, slopes=True)),
    "cap bias full": ("fp16", dict(softcap=30.0, slopes=True)),
    "docs": ("bf16", dict(causal=True, docs=True)),
    "docs full": ("fp16", dict(docs=True)),
    "docs cap": ("bf16", dict(causal=True, docs=True, softcap=30.0)),
    "docs cap running": ("fp16", dict(docs=True, softcap=30.0)),
    "docs bias": ("bf16", dict(causal=True, docs=True, slopes=True)),
    "docs bias full": ("fp16", dict(docs=True, slopes=True)),
    "prefix": ("bf16", dict(causal=True, prefix=True)),
    "prefix cap": ("bf16", dict(causal=True, prefix=True, softcap=30.0)),
    "prefix running": ("fp16", dict(causal=True, prefix=True, softcap=20.0)),
    "prefix bias": ("fp16", dict(causal=True, prefix=True, slopes=True)),
    "all": ("bf16", dict(causal=True, prefix=True, slopes=True, docs=True, softcap=15.0)),
}


def run_and_check(shape, D, form):
    B, H, Hkv, Sq, Skv = shape
    dt, kw = FORMS[form]
    kw = dict(kw)
    q, k, v = make(*shape, D, dt, 1)
    if kw.pop("docs", False):
        kw["doc_q"], kw["doc_k"] = documents(B, Sq, Skv)
    if kw.pop("slopes", False):
        # steep to flat: with the flat ones every tile counts
        kw["slopes"] = torch.logspace(0, -10, H, 2.0, device="cuda")
    if kw.pop("prefix", False):
        n = [Skv // 2, 129, 0, Skv + 50]
        kw["prefix"] = torch.tensor((n * B)[:B], dtype=torch.int32, device="cuda")
    o, lse = fa.fa_fwd_score(q, k, v, **kw)
    torch.cuda.synchronize()
    assert fa.fa_get_device_status() == fa.FA_OK
    seen, dist = ops_ref.score_seen(Sq, Skv, kw.get("causal", False), kw.get("prefix"),
                                    kw.get("doc_q"), kw.get("doc_k"))
    ref = ops_ref.attention(q, k, v, seen, D ** -0.5, kw.get("softcap", 0.0), kw.get("slopes"), dist,
                            p_step=torch.finfo(q.dtype).eps / 2)
    ops_ref.check(o, lse, ref)


WHOLE = [
    (1, 152, 76, 200, 400),   # one item an SM, a second stage of 72 rows, fewer tiles in stage 0
    (1, 80, 40, 513, 640),    # items of 256 rows and one of a single row
    (3, 100, 50, 513, 700),   # several items to a CTA
    (1, 90, 45, 513, 300),    # rows before key 0
]


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("shape", WHOLE, ids=lambda s: "x".join(map(str, s)))
def test_items_of_256_rows(shape, D, form):
    assert fa.fa_score_item_rows(*shape, D) == 256 and fa.fa_score_key_ranges(*shape, D) == 1
    run_and_check(shape, D, form)


SPLIT = [
    (1, 8, 4, 129, 1500),     # a range a tile, a second stage of one row
    (1, 30, 15, 200, 3000),
    (1, 1, 1, 4096, 16384),   # a chunk of one head's long prompt
]


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("shape", SPLIT, ids=lambda s: "x".join(map(str, s)))
def test_items_of_256_rows_with_split_keys(shape, D, form):
    assert fa.fa_score_item_rows(*shape, D) == 256 and fa.fa_score_key_ranges(*shape, D) > 1
    run_and_check(shape, D, form)


HALVES = [(11, 32, 16, 300, 300), (8, 16, 8, 800, 800), (2, 8, 4, 1021, 1500)]


@pytest.mark.parametrize("form", ["bias full", "cap bias full", "docs bias full", "docs", "all"])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("shape", HALVES, ids=lambda s: "x".join(map(str, s)))
def test_items_of_128_rows(shape, D, form):
    assert fa.fa_score_item_rows(*shape, D) == 128 and fa.fa_score_key_ranges(*shape, D) == 1
    run_and_check(shape, D, form)


def test_items_of_256_rows_take_the_prefill_kernels_sums():
    """Stage 0 with fewer tiles than stage 1, unmodified: the same bits."""
    for shape, D in (((1, 152, 152, 200, 400), 64), ((3, 100, 100, 513, 700), 128)):
        assert fa.fa_score_item_rows(*shape, D) == 256
        q, k, v = make(*shape, D, "bf16", 2)
        for causal in (False, True):
            a, b = fa.fa_fwd_ex(q, k, v, causal=causal, flags=fa.FA_FLAG_SINGLE_CTA, num_splits=1)
            o, lse = fa.fa_fwd_score(q, k, v, causal=causal)
            assert torch.equal(o, a) and torch.equal(lse, b)


def test_sizes_that_a_call_refuses_have_no_plan():
    for bad in ((0, 1, 1, 1, 1, 64), (1, 4, 3, 8, 8, 64), (1, 1, 1, 1, 1, 96), (1, 1, 1, 0, 1, 64)):
        assert fa.fa_score_item_rows(*bad) == 0 and fa.fa_score_key_ranges(*bad) == 0
