"""The calls that need libfp8lm.so alone work where the C++ module is missing or was built
for another PyTorch; those that need it say so."""
import subprocess
import sys
import textwrap

from conftest import ROOT


def run(body):
    head = """
        import sys
        sys.modules["fp8_gemms_b200._native"] = None    # importing it raises ImportError
        from fp8_gemms_b200 import api
    """
    return subprocess.run([sys.executable, "-c", textwrap.dedent(head) + textwrap.dedent(body)],
                          cwd=ROOT, capture_output=True, text=True)


def test_the_rest_of_the_api_is_there():
    r = run("""
        import torch
        assert api.Linear and api.Relu2Mlp and api.cast and api.LmError
        try:
            api.cast(torch.zeros(4, 16))       # refused by its own checks, not by an import
        except ImportError:
            raise SystemExit("cast needs the module")
        except Exception:
            pass
        freq, _ = api.rope_frequencies(8, device="cpu")
        assert freq.tolist()[0] == 1.0
    """)
    assert r.returncode == 0, r.stderr


def test_the_calls_that_need_it_say_so():
    r = run("""
        import torch
        x, rng = torch.zeros(4, 16), torch.zeros(2, dtype=torch.int64)
        calls = [lambda: api.layernorm(x), lambda: api.layernorm_backward(x, x, None, x[0], x[0]),
                 lambda: api.dropout_add(x, 0.1, rng), lambda: api.dropout_add_backward(x, 0.1, rng),
                 lambda: api.dropout_add_layernorm(x, x, None, None, 0.1, rng),
                 lambda: api.dropout_add_layernorm_backward(x, x, x, None, x[0], x[0], 0.1, rng),
                 lambda: api.rope([x], None), lambda: api.rope_backward([x], None)]
        for call in calls:
            try:
                call()
            except ImportError as e:
                assert "fp8_gemms_b200.build" in str(e) and "_native" in str(e), e
            else:
                raise SystemExit("no error")
    """)
    assert r.returncode == 0, r.stderr
