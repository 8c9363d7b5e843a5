"""Warp-wide instructions of the kernels on the paged cache stand where the warp is together.

mma.sync, movmatrix, tcgen05.ld and .st and their waits, TMEM's allocation and barriers of some of a block's threads have
.aligned forms: every lane of the warp has to execute the same one.  After code that only some lanes run (a branch, loop
or wait on a lane's own values) nothing but a warp-wide synchronisation says that the lanes are together again.  That
cannot be shown by running it, so the sources are read: each kernel statement by statement, the functions and lambdas
that it calls with it, loops twice.  A condition is taken for a lane's own unless every name in it is listed as one that
is the same for the whole warp."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "gated_deltanet_mixer_gb300", "csrc")
MEET = {"__syncwarp", "__syncthreads", "__any_sync", "__all_sync", "__ballot_sync"}
KEYWORDS = set("if else for while do switch return sizeof static_cast reinterpret_cast const constexpr true false nullptr int uint32_t "
               "uint64_t float auto min max long bool void unsigned asm volatile".split())
NAME = re.compile(r"[A-Za-z_]\w*")
LAMBDA = re.compile(r"\[[&=\w, ]*\]\s*(\([^()]*(\([^()]*\)[^()]*)*\))?\s*(->\s*\w+\s*)?$")
CONSTANT = re.compile(r"k[A-Z]\w*$|[A-Z]\w{0,2}$")  # kThreads; D, NT, SUB


def clean(text):
    """Without comments and preprocessor lines; quoted text without what would look like code's structure."""
    text = re.sub(r"//[^\n]*", "", text)
    text = re.sub(r"(?m)^[ \t]*#(.*\\\n)*.*$", "", text)
    return re.sub(r'"(\\.|[^"\\\n])*"', lambda m: re.sub(r"[{}();,\[\]]", " ", m.group(0)), text)


class Reader:
    """Statements: ("if", condition, then, else, line), ("loop", head, body, line), ("block", statements),
    ("text", text, lambdas, line) with lambdas as (name, statements)."""

    def __init__(self, text):
        self.s, self.i, self.functions = clean(text), 0, {}
        self.declarations()

    def line(self, i=None):
        return self.s.count("\n", 0, self.i if i is None else i) + 1

    def space(self):
        while self.i < len(self.s) and self.s[self.i].isspace():
            self.i += 1

    def close(self, i):
        """Behind the bracket that closes the one at i."""
        depth = 0
        for j in range(i, len(self.s)):
            depth += (self.s[j] in "({[") - (self.s[j] in ")}]")
            if depth == 0:
                return j + 1
        raise ValueError("unbalanced")

    def declarations(self):
        """Functions (methods too) of a file, namespace or structure; up to a closing brace."""
        start = self.i
        while self.i < len(self.s):
            ch = self.s[self.i]
            if ch == "}":
                self.i += 1
                return
            if ch == ";":
                start = self.i + 1
            if ch == "(":
                self.i = self.close(self.i)
                continue
            if ch == "{":
                head = self.s[start:self.i]
                plain = re.sub(r"__launch_bounds__\s*\([^()]*(\([^()]*\)[^()]*)*\)", "", head)
                name = re.search(r"(\w+)\s*\(", plain)
                if re.match(r"\s*(inline )?\s*namespace\b", head) or re.search(r"\bstruct\b[^()=]*$", head):
                    self.i += 1
                    self.declarations()
                elif name and "=" not in plain.split("(")[0]:
                    begin = self.i
                    self.i += 1
                    body = self.statements()
                    self.functions[name.group(1)] = (body, "__global__" in head, ".aligned" in self.s[begin:self.i])
                else:
                    self.i = self.close(self.i)
                start = self.i
                continue
            self.i += 1

    def statements(self):
        out = []
        while True:
            self.space()
            if self.s[self.i] == "}":
                self.i += 1
                return out
            out.append(self.statement())

    def statement(self):
        self.space()
        line = self.line()
        if self.s[self.i] == "{":
            self.i += 1
            return ("block", self.statements())
        word = NAME.match(self.s, self.i)
        word = word.group(0) if word else ""
        if word in ("if", "for", "while", "switch"):
            self.i += len(word)
            self.space()
            constexpr = self.s.startswith("constexpr", self.i)
            if constexpr:
                self.i += len("constexpr")
                self.space()
            end = self.close(self.i)
            head = self.s[self.i + 1:end - 1]
            self.i = end
            body = self.statement()
            if word != "if":
                return ("loop", head, body, line)
            self.space()
            other = None
            if re.match(r"else\b", self.s[self.i:]):
                self.i += 4
                other = self.statement()
            return ("if", "" if constexpr else head, body, other, line)
        text, lambdas = "", []
        while self.s[self.i] != ";":
            ch = self.s[self.i]
            if ch == "{":
                if LAMBDA.search(text):
                    name = re.findall(r"(\w+)\s*=", text) or [""]
                    self.i += 1
                    lambdas.append((name[-1], self.statements()))
                    text = LAMBDA.sub("", text)
                    continue
                end = self.close(self.i)
                text += self.s[self.i:end]
                self.i = end
                continue
            text += ch
            self.i += 1
        self.i += 1
        return ("text", text, lambdas, line)


class Check:
    def __init__(self, functions, aligned, uniform):
        self.functions, self.aligned, self.uniform, self.bad = dict(functions), aligned, uniform, set()

    def same(self, condition):
        """Whether a condition is the same for the warp: votes are, whatever of."""
        text = condition
        for vote in ("__any_sync", "__all_sync", "__ballot_sync"):
            while vote in text:
                i = text.index(vote)
                depth, j = 0, text.index("(", i)
                for j in range(j, len(text)):
                    depth += (text[j] == "(") - (text[j] == ")")
                    if depth == 0:
                        break
                text = text[:i] + "0" + text[j + 1:]
        text = re.sub(r"(\.|->|::)\s*\w+", "", re.sub(r"\b0x[0-9a-fA-F]+u?\b|\b\d[\w.]*", "0", text))
        return all(n in KEYWORDS or n in self.uniform or CONSTANT.match(n) for n in NAME.findall(text))

    def text(self, text, state, apart, line):
        for m in re.finditer(r"([A-Za-z_]\w*)\s*(<[^;=]*?>)?\s*\(", text):
            name = m.group(1)
            if name in MEET:
                state = not apart
            elif name in self.aligned:
                if not state:
                    self.bad.add(line)
            elif name in self.functions:
                body = self.functions.pop(name)  # none calls itself
                before = set(self.bad)
                state = self.run(body, state, apart)
                if self.bad - before:
                    self.bad.add(line)
                self.functions[name] = body
        return state

    def run(self, node, state, apart=False):
        """Whether the warp is together behind the node; apart: only some lanes are here."""
        if isinstance(node, list):
            known = dict(self.functions)
            for n in node:
                state = self.run(n, state, apart)
            self.functions = known
            return state
        if node[0] == "block":
            return self.run(node[1], state, apart)
        if node[0] == "text":
            for name, body in node[2]:
                self.functions[name] = body
            state = self.text(node[1], state, apart, node[3])
            return state and not (apart and re.match(r"\s*(return|break|continue)\b", node[1]))
        if node[0] == "if":
            state = self.text(node[1], state, apart, node[4])
            same = self.same(node[1])
            out = self.run(node[2], state and same, apart or not same)
            other = self.run(node[3], state and same, apart or not same) if node[3] else state
            return same and out and other
        same = self.same(node[1])
        state = self.text(node[1], state, apart, node[3])
        once = self.run(node[2], state and same, apart or not same)
        again = self.run(node[2], state and same and once, apart or not same)
        return same and state and once and again


def unsafe(name, uniform, path=CSRC, text=None):
    """Lines of the kernels of a file with an aligned instruction that lanes may reach apart (and those of the calls)."""
    headers = {}
    for h in ("umma.cuh", "cache_device.cuh"):
        with open(os.path.join(CSRC, h)) as f:
            headers.update(Reader(f.read()).functions)
    if text is None:
        with open(os.path.join(path, name)) as f:
            text = f.read()
    own = Reader(text).functions
    every = {**headers, **own}
    aligned = {n for n, (_, _, a) in every.items() if a and n not in own} | {n for n, (_, g, a) in own.items() if a and not g}
    kernels = {n: b for n, (b, g, _) in own.items() if g}
    assert kernels
    check = Check({n: b for n, (b, g, a) in every.items() if not g and n not in aligned}, aligned | {"sync"}, uniform)
    for body in kernels.values():
        check.run(body, True)
    return sorted(check.bad)


# Names in conditions and loops that are the same for all lanes of a warp.
FILES = {
    "attn_few.cu": set("ch e i i2 j k masked mine s u upper".split()),
    "attn_tile.cu": set("d group h i j ntiles split warp".split()),
    "kv_append.cu": set(),
    "kv_pages.cu": set("a b0 blockDim".split()),
}


@pytest.mark.parametrize("name", sorted(FILES))
def test_aligned_instructions_stand_where_the_warp_is_together(name):
    assert unsafe(name, FILES[name]) == []


HEAD = "namespace x {\n__device__ void mma(int k) { asm(\"mma.sync.aligned\"); }\n__global__ void f(int n) {\nint lane = threadIdx.x;\n"


def lines(body):
    return [n - HEAD.count("\n") for n in unsafe("", {"n", "i"}, text=HEAD + body + "\n}\n}\n") if n > HEAD.count("\n")]


def test_the_reading_itself():
    assert lines("mma(0);") == []
    assert lines("if (lane < n) store();\nmma(0);") == [2]
    assert lines("if (lane < n) store();\n__syncwarp();\nmma(0);") == []
    assert lines("if (lane < n) mma(0);") == [1]
    assert lines("if (lane < n) {\n__syncwarp();\nmma(0);\n}") == [3]          # not a meeting of all
    assert lines("if (n > 3) {\nif (lane) store();\n__syncwarp();\n}\nmma(0);") == []
    assert lines("if (lane) store();\nif (n > 3) __syncwarp();\nmma(0);") == [3]
    assert lines("if (n > 3)\nfor (int i = 0; i < n; ++i)\nif (lane > i) x[i] = 0;\nmma(0);") == [4]
    assert lines("for (int i = 0; i < n; ++i) {\nmma(0);\nif (lane) store();\n}") == [2]  # round the loop
    assert lines("for (int i = 0; i < n; ++i) {\n__syncwarp();\nmma(0);\nif (lane) store();\n}") == []
    assert lines("for (int i = lane; i < n; i += 32) store();\nmma(0);") == [2]
    assert lines("auto wait = [&](int b) {\nif (ready(b)) return;\nspin();\n};\nwait(0);\nmma(0);") == [6]
    assert lines("auto go = [&] { mma(0); };\nif (lane) store();\ngo();") == [1, 3]
    assert lines("if (__any_sync(~0u, lane > n)) mma(0);") == []
    assert lines("x = lane > n ? 0 : x;  // if (lane)\nmma(0);") == []
