"""What the binding of the serving calls gives back: tensors of their own, and
the library's status for what it refuses."""

import pytest
import torch

import dequant_gemv_rht_amd as dq

pytestmark = pytest.mark.gpu


def i32(*v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def slots(tokens=5, **kw):
    args = dict(page_size=16, pages=9, table=torch.full((2, 3), -1, dtype=torch.int32, device="cuda"), lens=i32(0, 0),
                new_tokens=i32(3, 2), free_pages=i32(4, 5, 6), used=i32(0), tokens=tokens)
    return dq.wq_kv_slots(**{**args, **kw})


WANT = [[64, 65, 66, 80, 81], [0, 1, 2, 0, 1], [0, 0, 0, 1, 1], [3, 2], [2, 4], [2]]


@pytest.mark.parametrize("which", range(6))
def test_slots_outputs_do_not_share_memory(which):
    """One output that grows leaves the others alone."""
    got = slots()
    assert [t.tolist() for t in got] == WANT
    assert len({t.untyped_storage().data_ptr() for t in got}) == 6
    assert all(t.storage_offset() == 0 and t.untyped_storage().nbytes() == t.nbytes for t in got)
    got[which].resize_(40).fill_(-9)
    assert [t.tolist() for i, t in enumerate(got) if i != which] == [w for i, w in enumerate(WANT) if i != which]


@pytest.mark.parametrize("tokens", [(1 << 30) + 1, 1 << 40, 1 << 61, 1 << 62, (1 << 63) - 1])
def test_slots_of_too_many_rows_are_refused_before_any_memory(tokens):
    table, lens, free, used = torch.full((2, 3), -1, dtype=torch.int32, device="cuda"), i32(0, 0), i32(1), i32(0)
    before = torch.cuda.memory_stats()["allocation.all.allocated"]
    with pytest.raises(dq.WqError, match="tokens above 2") as e:
        dq.wq_kv_slots(16, 9, table, lens, lens, free, used, tokens)
    assert e.value.status == dq.WQ_E_UNSUPPORTED
    assert torch.cuda.memory_stats()["allocation.all.allocated"] == before


@pytest.mark.parametrize("rank,k,n,status,text", [(12, 128, 8, dq.WQ_E_UNSUPPORTED, "rank"), (136, 128, 8, dq.WQ_E_UNSUPPORTED, "rank"),
                                                  (8, 192, 8, dq.WQ_E_ARG, "128"), (8, 128, 0, dq.WQ_E_ARG, "n=0")])
def test_status_of_refused_adapters(rank, k, n, status, text):
    half = lambda *s: torch.zeros(s, dtype=torch.float16, device="cuda")  # noqa: E731
    with pytest.raises(dq.WqError, match=text) as e:
        dq.wq_lora([half(2, rank, k)], [half(2, n, rank)], [half(3, k)], i32(0, 1, 1), [half(3, n)])
    assert e.value.status == status


@pytest.mark.parametrize("vocab,status,text", [(0, dq.WQ_E_ARG, "vocab=0"), ((1 << 20) + 1, dq.WQ_E_UNSUPPORTED, "2^20")])
def test_status_of_refused_sampling(vocab, status, text):
    with pytest.raises(dq.WqError) as e:
        dq.wq_sample(torch.zeros((2, vocab), device="cuda"), torch.zeros(2, device="cuda"))
    assert e.value.status == status and text in str(e.value)
