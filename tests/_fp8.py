"""Which kernel an 8-bit product goes to, by the library's own rule: read from its source, so that a test that wants the
tiles of many rows fails when the rule moves its sizes elsewhere."""
import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "sparse_gemm_b200", "csrc")


def _returned(file, function):
    text = open(os.path.join(CSRC, file)).read()
    return re.search(rf"\b{function}\([^)]*\)\s*\{{\s*return ([^;]*);", text).group(1)


def _python(expression):
    expression = re.sub(r"static_cast<int64_t>", "", expression)
    expression = re.sub(r"\b(\d+)ll\b", r"\1", expression)
    return expression.replace("||", " or ").replace("&&", " and ").replace("num_sms()", "148")


def kernel_of(T, E, cols, transposed=False):
    """'rows8' (up to eight rows), 'few' or 'many' for a product of T rows with `cols` output columns."""
    names = dict(T=T, E=E, cols=cols, kRows=8, kMostRows=64,
                 most_tiles=lambda T, E, cols: -(-cols // 128) * (min(T, E) + T // 64))
    if not transposed and eval(_python(_returned("few_rows.cu", "few_rows8")), names):
        return "rows8"
    return "few" if eval(_python(_returned("fp8_few.cu", "fp8_few")), names) else "many"
