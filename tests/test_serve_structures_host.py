"""Host side of the serving operators: sizes that their C structures cannot hold are refused in words."""
import pytest

from gated_delta_rule_54_gb300 import serve

BIG = 1 << 31


@pytest.mark.parametrize("pack,fields", [
    (serve._KV8, [1, 2, 3, BIG, 5, 6, 7, 64, 16, 1, 0, 1, 9, 0.5, 4096, *range(8, 56, 8)]),      # tokens
    (serve._KV8, [1, 2, 3, 4, 5, 6, 7, 64, 16, 1, 0, 1, BIG, 0.5, 4096, *range(8, 56, 8)]),      # window
    (serve._KV8, [1, 2, 3, 4, 5, 6, 7, 64, 16, 1, 0, 1, 9, "a", 4096, *range(8, 56, 8)]),        # scale
    (serve._POOL, [1, 2, BIG, 4, 5, 6, 7]),                                                      # columns
    (serve._BEAM, [1, 2, 3, BIG, 5, 6, 7]),                                                      # vocabulary
    (serve._BEAM, [1, 2, 3, 4, 5, 6, -BIG - 1]),                                                 # eos
    (serve._ROTARY, [1, 2, 3, 4, BIG, 0]),                                                       # dims that turn
    (serve._LOGITS, [1, 2, 3, 4, BIG, 6, 7]),                                                    # vocabulary
    (serve._LOGITS, [1, 2, 3, 4, 5, BIG, 7]),                                                    # columns
])
def test_sizes_beyond_the_structure_are_refused_in_words(pack, fields):
    with pytest.raises(ValueError, match="does not fit"):
        pack(*fields)
