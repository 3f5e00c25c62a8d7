"""A commit or an eviction of caches held in 8 or 4 bits takes K and V of the same rows: the
rows of one are moved by the other's size, which would reach past a smaller cache."""
import pytest
import torch

import speculative_decoding_verification_masked_gb300 as va


def cache(nbytes, tokens=8, dtype=torch.uint8):
    return torch.zeros(1, tokens, 2, nbytes, dtype=dtype)


I32 = torch.zeros(1, dtype=torch.int32)
PATH = torch.zeros(1, 4, dtype=torch.int32)
TABLE = torch.zeros(1, 1, dtype=torch.int32)
IDX, N = torch.zeros(1, 2, 4, dtype=torch.int32), torch.zeros(1, 2, dtype=torch.int32)


@pytest.mark.parametrize("k,v", [(cache(144), cache(80)), (cache(80), cache(144)), (cache(80), cache(40, dtype=torch.bfloat16)),
                                 (cache(64, dtype=torch.bfloat16), cache(80)), (cache(80), cache(80, 7))])
def test_k_and_v_of_different_rows(k, v):
    for call in (lambda: va.verify_commit_kv_dense(k, v, I32, PATH, I32),
                 lambda: va.verify_commit_kv_paged(k, v, TABLE, I32, PATH, I32),
                 lambda: va.verify_evict_kv_dense(k, v, I32, IDX, N),
                 lambda: va.verify_evict_kv_paged(k, v, TABLE, I32, IDX, N)):
        with pytest.raises(ValueError, match="same rows"):
            call()
