"""The attention entry points' host checks at their edges, without a GPU."""
import pytest

from tests.test_attention_cpu import EINVAL, ENODEV, OK, P, batch, no_gpu, prompt


@no_gpu
@pytest.mark.parametrize("unused", [dict(block_table=None), dict(bt_stride=0), dict(block_table=None, bt_stride=-5),
                                    dict(num_blocks=0)], ids=str)
def test_packed_prompts_need_no_block_table(unused):
    # accepted: it reaches the device, of which there is none
    assert prompt(b=batch(**unused), start=P(256)) == ENODEV


def test_prompts_in_pages_need_their_block_table():
    for bad in (dict(block_table=None), dict(bt_stride=0), dict(num_blocks=49)):
        assert prompt(b=batch(**bad)) == EINVAL, bad
    # what packed keys need all the same
    for bad in (dict(query_start_loc=None), dict(seq_lens=None), dict(max_seq_len=-1), dict(num_reqs=-1)):
        assert prompt(b=batch(**bad), start=P(256)) == EINVAL, bad
    assert prompt(b=batch(num_decodes=3, num_decode_tokens=12, block_table=None), start=P(256)) == OK  # no rows
