"""profiles/traffic.py: the bytes of an ncu CSV, under the hash of the sources as they are when it
runs, so that bench.py reports them for those sources and no others."""
import importlib.util
import json
import os

import bench

HERE = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEAD = '"ID","Kernel Name","Metric Name","Metric Unit","Metric Value"\n'
CSV = ["==PROF== Connected\n", HEAD,
       '"0","void fwd::fa_fwd_kernel<128, 0, 0, 0, 0>(CUtensorMap_st, fwd::Params)","dram__bytes_read.sum","byte","1,000"\n',
       '"0","void fwd::fa_fwd_kernel<128, 0, 0, 0, 0>(CUtensorMap_st, fwd::Params)","dram__bytes_write.sum","byte","24"\n',
       '"0","void fwd::fa_fwd_kernel<128, 0, 0, 0, 0>(CUtensorMap_st, fwd::Params)","gpu__time_duration.sum","ns","7"\n',
       '"1","bwd::fa_bwd_kernel(Params)","dram__bytes_read.sum","byte","10"\n',
       '"2","bwd::fa_bwd_kernel(Params)","dram__bytes_read.sum","byte","30"\n']


def _script():
    spec = importlib.util.spec_from_file_location("traffic", os.path.join(HERE, "profiles", "traffic.py"))
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


def test_bytes_and_hash(monkeypatch, tmp_path):
    t = _script()
    assert t.bytes_per_launch(CSV) == {"fa_fwd_kernel": 1024, "fa_bwd_kernel": 20}
    table = t.record("w", "profiles/x.md", CSV)
    assert {e["source_sha"] for e in table.values()} == {bench.kernel_source_sha()}
    (tmp_path / "profiles").mkdir()
    (tmp_path / "profiles" / "traffic.json").write_text(json.dumps(table))
    monkeypatch.setattr(bench, "ROOT", str(tmp_path))
    monkeypatch.setattr(bench, "kernel_source_sha", lambda: table["fa_fwd_kernel"]["source_sha"])
    assert bench.profiled_traffic("fa_fwd_kernel", "w") == 1024
    monkeypatch.setattr(bench, "kernel_source_sha", lambda: "other sources")
    assert bench.profiled_traffic("fa_fwd_kernel", "w") is None
