"""A workspace made for the largest batch serves the smaller ones: no size is above that of more tokens or rows."""
import pytest


@pytest.fixture(scope="module")
def L():
    from gemm_q1_q8_gb300 import build
    build.build()
    import gemm_q1_q8_gb300 as gq
    return gq.lib()


@pytest.mark.parametrize("type_", [0, 1, 2])
@pytest.mark.parametrize("rows,n", [(1, 128), (32, 1 << 20), (64, 256), (129, 640), (2560, 2560), (2560, 6912), (6912, 2560), (9856, 4096), (14336, 4096),
                                    (38912, 1024), (49152, 2560)])
def test_products(L, rows, n, type_):
    sizes = [L.gq_q1_q8_linear_workspace_bytes(rows, n, m, type_) for m in list(range(1, 1300)) + [4096, 65536, 1 << 20]]
    assert all(0 < a <= b for a, b in zip(sizes, sizes[1:]))
    # not much above what the activations' parts take
    assert all(s <= 4 * m * n + 4 * m + 512 + 152 * 2 * 128 * 128 * 4 for m, s in enumerate(sizes[:1299], 1))


@pytest.mark.parametrize("vocab", [1, 33, 49152, 262144, 262145, 300001, 600000, 1 << 20])
def test_log_probabilities(L, vocab):
    most = min(vocab, 32)
    tops = [[L.gq_logprobs_workspace_bytes(m, vocab, k) for m in list(range(1, 400)) + [4096, 1 << 24]] for k in range(most + 1)]
    for sizes in tops:
        assert all(16 <= a <= b for a, b in zip(sizes, sizes[1:]))
    for fewer, more in zip(tops, tops[1:]):
        assert all(a <= b for a, b in zip(fewer, more))
