"""What all calls of the dense side share: the device's status word, the current
device, gradients."""
import threading

import pytest
import torch

import dlrm_sparse_embedding_gb300 as emb

gpu = pytest.mark.gpu


@gpu
@pytest.mark.parametrize("callers", [2, 8, 100])
def test_of_many_callers_one_gets_the_status(callers):
    ids = torch.tensor([[0], [9]], dtype=torch.int32, device="cuda")
    streams = [torch.cuda.Stream() for _ in range(callers)]
    for _ in range(200 if callers < 100 else 10):
        emb.expert_sort(ids, 4)
        torch.cuda.synchronize()
        begin, got = threading.Barrier(callers), [None] * callers

        def ask(i):
            begin.wait()
            got[i] = emb.dense_status(streams[i])

        threads = [threading.Thread(target=ask, args=(i,)) for i in range(callers)]
        for t in threads:
            t.start()
        for t in threads:
            t.join()
        assert sorted(got) == sorted([emb.EMB_ERR_KEY_RANGE] + [emb.EMB_OK] * (callers - 1))
