"""How the attention's work is cut, as far as the size of its workspace tells:
256 bytes for a workgroup per unit, more where contexts may be split. No GPU."""
import pytest

from draft_verify_sampling_spec_amd import binding as sb


def _split(B, K, Hq, Hkv, D, pages, window=0, page=64):
    return sb.spec_verify_attention_workspace_bytes(B, K, Hq, Hkv, D, page, pages, window) > 256


@pytest.mark.parametrize("B,K,Hq,Hkv,D", [(128, 5, 24, 8, 256), (512, 2, 16, 8, 128), (1024, 2, 16, 8, 64),
                                          (16384, 0, 8, 8, 128)])
def test_many_units_split_where_one_request_may_be_much_longer_than_the_others(B, K, Hq, Hkv, D):
    """Many units even out by themselves only if none of them can be long."""
    assert not _split(B, K, Hq, Hkv, D, 8)
    assert not _split(B, K, Hq, Hkv, D, 32)
    assert _split(B, K, Hq, Hkv, D, 4096 if B < 16384 else 1 << 18)
    # A window bounds every request's span.
    assert not _split(B, K, Hq, Hkv, D, 4096, window=1500)


def test_few_units_split_unless_all_are_short():
    assert _split(1, 4, 32, 8, 128, 2048)
    assert not _split(1, 4, 32, 8, 128, 8)
    assert _split(128, 8, 32, 8, 128, 128)
