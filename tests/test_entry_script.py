"""__graft_entry__.py as a program: its last statement runs what stands above it."""
import os
import runpy
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_everything_is_defined_when_the_program_runs(monkeypatch):
    """`python __graft_entry__.py`, with the compiler left out: by the time build() is called, every
    function of the file that smoke() needs is there."""
    from mla_decode_attention_folded_gb300 import build
    path = os.path.join(ROOT, "__graft_entry__.py")
    monkeypatch.setattr(sys, "argv", [path])
    seen = []

    def compiled():
        frame = sys._getframe(1)                   # build() of the program
        seen.append(set(frame.f_globals))

    monkeypatch.setattr(build, "build", compiled)
    names = runpy.run_path(path, run_name="__main__")
    functions = {n for n, f in names.items() if callable(f) and getattr(f, "__module__", "") == "__main__"}
    assert {"smoke", "_smoke_step", "_smoke_cache", "_smoke_prompt"} <= functions
    assert len(seen) == 1 and functions <= seen[0], f"not yet defined: {functions - seen[0]}"
