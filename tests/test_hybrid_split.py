"""Which requests the absorbed attention's second kernel joins, checked on the host
(tests/latent_joins_host.cu)."""
import os
import subprocess

from kimi_delta_attention_07_gb300 import _build


def test_every_request_that_crosses_a_range_has_one_record(tmp_path):
    source = os.path.join(os.path.dirname(os.path.abspath(__file__)), "latent_joins_host.cu")
    program = str(tmp_path / "latent_joins_host")
    subprocess.run([_build.nvcc(), "-std=c++17", "-O1", "--expt-relaxed-constexpr", "-I", _build.INCLUDE, "-I", _build.CSRC,
                    source, "-o", program], check=True)
    out = subprocess.run([program], capture_output=True, text=True, timeout=120).stdout
    assert out.startswith("ok ") and int(out.split()[1]) > 3000, out


def test_only_the_first_row_block_writes_records():
    """One writer, which no failed wait reaches: a record that another row block took back would leave healthy rows unwritten."""
    with open(os.path.join(_build.CSRC, "kda_latent_decode.cu")) as f:
        source = f.read()
    assert source.count("write_joins(") == 1 and "p.joins[" not in source.replace("p.joins[blockIdx.x]", "")
