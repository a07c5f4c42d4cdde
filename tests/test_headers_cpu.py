"""The C headers as a C or C++ program takes them: each compiles by itself with
the headers that it names and no others, ngram.h and ssm.h with none."""
import os
import shutil
import subprocess

import pytest

INCLUDE = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include")
CALL = """
#include "ngram.h"
#include "drop.h"
int f(const ngram_config *c, const drop_spec *s, void *p) { return ngram_embed_fwd_drop(c, p, p, 0, 0, s, p, p, p); }
"""


def _compile(path, lang):
    cc = {"c": ["gcc", "-std=c11"], "c++": ["g++", "-std=c++17"]}[lang]
    r = subprocess.run([*cc, "-x", lang, "-Wall", "-Wextra", "-pedantic", "-Werror", "-fsyntax-only", path],
                       capture_output=True, text=True)
    assert r.returncode == 0, r.stderr


@pytest.mark.parametrize("lang", ["c", "c++"])
@pytest.mark.parametrize("header,needs", [("ngram.h", []), ("ssm.h", []), ("drop.h", []), ("ffn.h", ["drop.h"])])
def test_header_stands_alone(tmp_path, header, needs, lang):
    for h in [header, *needs]:
        shutil.copy(os.path.join(INCLUDE, h), tmp_path)
    src = tmp_path / "use.c"
    src.write_text(f'#include "{header}"\n#include "{header}"\nint unused;\n')
    _compile(str(src), lang)


@pytest.mark.parametrize("lang", ["c", "c++"])
@pytest.mark.parametrize("order", ["as is", "reversed"])
def test_dropped_forward_with_both_headers(tmp_path, order, lang):
    for h in ("ngram.h", "drop.h"):
        shutil.copy(os.path.join(INCLUDE, h), tmp_path)
    text = CALL
    if order == "reversed":
        text = text.replace('"ngram.h"', '"x"').replace('"drop.h"', '"ngram.h"').replace('"x"', '"drop.h"')
    src = tmp_path / "use.c"
    src.write_text(text)
    _compile(str(src), lang)
