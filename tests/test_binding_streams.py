"""What a call of the binding makes for itself - its error word, workspace and
outputs - is made on the stream that the call was given (read from the source;
no GPU needed)."""
import ast
import os

import dropless_grouped_gemm_gb300 as M

MAKERS = {"_err_word": 2, "_scratch": 2, "_workspace": 3, "_empty": 3}      # name: position of the stream


def _calls():
    """(function, call) of every call of a maker inside a function with a
    `stream` parameter."""
    tree = ast.parse(open(os.path.join(os.path.dirname(M.__file__), "__init__.py"), encoding="utf-8").read())
    for f in tree.body:
        if isinstance(f, ast.FunctionDef) and not f.name.startswith("_"):
            names = {a.arg for a in f.args.args + f.args.kwonlyargs}
            if "stream" in names:
                yield from ((f.name, c) for c in ast.walk(f) if isinstance(c, ast.Call))


def test_what_a_call_makes_takes_its_stream():
    missing = []
    for name, c in _calls():
        maker = getattr(c.func, "id", None)
        # torch's own allocations are in the current stream's memory
        if isinstance(c.func, ast.Attribute) and c.func.attr in ("empty", "zeros", "full", "ones", "empty_like",
                                                                 "zeros_like", "clone"):
            missing.append((name, c.lineno))
        if maker in MAKERS:
            given = list(c.args[MAKERS[maker]:]) + [k.value for k in c.keywords if k.arg == "stream"]
            if not any(isinstance(a, ast.Name) and a.id == "stream" for a in given):
                missing.append((name, c.lineno))
    assert not missing, missing
