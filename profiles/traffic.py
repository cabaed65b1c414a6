"""DRAM bytes per launch from an ncu CSV, as profiles/traffic.json holds them.

    python profiles/traffic.py <workload> <summary .md> <ncu csv> > traffic.json

Run it where and when the capture is taken: the source hash that it writes is that of the
kernels' sources at that moment, and bench.py reports the bytes only while it still holds.
"""
import csv
import json
import os
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, ROOT)

BYTES = ("dram__bytes_read.sum", "dram__bytes_write.sum")


def bytes_per_launch(lines):
    """{kernel: DRAM bytes read and written by a launch (the mean, of more than one)}."""
    rows = csv.DictReader(line for line in lines if line.startswith('"'))
    total, launches = {}, {}
    for r in rows:
        if r["Metric Name"] in BYTES:
            if r["Metric Unit"] != "byte":
                raise ValueError(f"{r['Metric Name']} in {r['Metric Unit']}: pass --print-units base")
            name = r["Kernel Name"].split("<")[0].split("(")[0].split("::")[-1].split()[-1]
            total[name] = total.get(name, 0) + int(r["Metric Value"].replace(",", ""))
            launches.setdefault(name, set()).add(r["ID"])
    return {name: total[name] // len(launches[name]) for name in sorted(total)}


def record(workload, summary, lines):
    from bench import kernel_source_sha

    sha = kernel_source_sha()
    return {name: {"workload": workload, "bytes_per_launch": n, "source_sha": sha, "from": summary}
            for name, n in bytes_per_launch(lines).items()}


if __name__ == "__main__":
    with open(sys.argv[3]) as f:
        table = record(sys.argv[1], sys.argv[2], f)
    if not table:
        sys.exit("no kernel with DRAM bytes in " + sys.argv[3])
    print(json.dumps(table, indent=1))
