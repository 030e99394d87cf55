"""Row lengths and counts beyond what the kernels' 32-bit channel indexes and 64-bit group counts hold are refused (CPU only)."""
import pytest

import gated_delta_rule_20_amd as kda

A = 0x10000  # an aligned address that nothing dereferences


@pytest.mark.parametrize("R,D,status", [
    (1, 0x7fffffff, 2), (4, 0x7fffffff - 127, 2), (1, (1 << 24) + 1, 2), (1 << 40, 0x7fffffff, 2),
    (1 << 40, 1 << 24, 2),                      # 2^57 groups
    (1 << 47, 1 << 24, 2), (0x7fffffffffffffff, 1, 2), (0x7fffffffffffffff, 1 << 24, 2),
])
def test_pack_and_unpack_refuse(R, D, status):
    lib = kda.load_library()
    assert lib.kda_act_unpack(1, A, A, R, D, A, None) == status
    assert "D" in lib.kda_last_error_message().decode()
    assert lib.kda_act_pack(1, A, D, R, D, A, A, None) == status
    assert "D" in lib.kda_last_error_message().decode()
