"""norm.h and recur.h as a C or C++ program takes them: alone, and together with
every other header."""
import os
import shutil

import pytest

from test_headers_cpu import INCLUDE, _compile

ALL = ["ngram.h", "ssm.h", "drop.h", "ffn.h", "norm.h", "recur.h"]


@pytest.mark.parametrize("lang", ["c", "c++"])
@pytest.mark.parametrize("headers", [["norm.h"], ["recur.h"], ALL, ALL[::-1]])
def test_headers(tmp_path, headers, lang):
    for h in headers:
        shutil.copy(os.path.join(INCLUDE, h), tmp_path)
    src = tmp_path / "use.c"
    src.write_text("".join(f'#include "{h}"\n' for h in headers * 2) + "int unused;\n")
    _compile(str(src), lang)
