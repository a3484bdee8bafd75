"""What the speculative decoder refuses before it touches a GPU."""

import pytest

from affine_quantized_gemm_amd import spec_decode as S


@pytest.mark.parametrize("args", [["--sinks", "4"], ["--window", "-1"], ["--window", "64", "--sinks", "-2"],
                                  ["--seqs", "10", "--depth", "4"]])
def test_arguments(args, capsys):
    with pytest.raises(SystemExit) as e:
        S.main(args)
    assert e.value.code == 2 and "error:" in capsys.readouterr().err


def test_sinks_without_a_window():
    with pytest.raises(ValueError, match="sinks need a window"):
        S.Decoder(sinks=4)
