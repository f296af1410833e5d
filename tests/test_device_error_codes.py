"""The codes that kernels store in the device error word: one enumeration, no code twice, each the
public status of the same name."""

import re
from pathlib import Path

import gated_delta_rule_144_b200 as kda

ROOT = Path(__file__).resolve().parent.parent
CSRC = ROOT / "gated_delta_rule_144_b200" / "csrc"


def enum(text, name):
    body = re.search(r"enum %s\s*(?::\s*\w+\s*)?\{(.*?)\}" % name, text, re.S).group(1)
    body = re.sub(r"/\*.*?\*/|//[^\n]*", "", body, flags=re.S)
    return {a: int(b) for a, b in re.findall(r"(\w+)\s*=\s*(\d+)", body)}


def test_device_codes_are_public_statuses():
    device = enum((CSRC / "kda_internal.cuh").read_text(), "DeviceError")
    text = (ROOT / "include" / "kda.h").read_text()
    public = next({a: int(b) for a, b in re.findall(r"(KDA_(?:OK|ERR_\w+)) = (\d+)", body)}
                  for body in re.findall(r"typedef enum \{(.*?)\} kda_status_t", text, re.S))
    assert len(set(device.values())) == len(device) and len(set(public.values())) == len(public)
    for name, code in device.items():
        assert public[name.replace("DEV_", "KDA_" if code == 0 else "KDA_ERR_")] == code
    assert {v: k for k, v in public.items()} == kda.STATUS
    used = set()
    for f in CSRC.glob("*.cu*"):
        text = f.read_text()
        used |= set(re.findall(r"\bDEV_[A-Z_]+\b", text))
        if f.name != "kda_internal.cuh":   # declared nowhere else
            assert not re.search(r"\bDEV_[A-Z_]+\s*=(?!=)", text), f.name
    assert used <= set(device)
