// status_check.cu -- host-only check of the status words' read: the runtime's
// calls are stand-ins that count.  Prints "ok <cases>" or the first violation.
#include <cuda_runtime.h>

#include <cstdio>
#include <cstdlib>

static unsigned int g_word;
static int g_reads, g_writes, g_waits, g_fail_at, g_calls;

static cudaError_t step() { return ++g_calls == g_fail_at ? cudaErrorUnknown : cudaSuccess; }
static cudaError_t read_word(unsigned int *out) {
    ++g_reads;
    *out = g_word;
    return step();
}
static cudaError_t write_word(const unsigned int *in) {
    ++g_writes;
    g_word = *in;
    return step();
}
static cudaError_t wait() {
    ++g_waits;
    return step();
}

#define cudaMemcpyFromSymbolAsync(out, word, n, at, kind, stream) read_word(out)
#define cudaMemcpyToSymbolAsync(word, in, n, at, kind, stream) write_word(in)
#define cudaStreamSynchronize(stream) wait()
#include "status.cuh"

#define REQUIRE(c)                               \
    do {                                         \
        if (!(c)) {                              \
            std::printf("violation: %s\n", #c);  \
            std::exit(1);                        \
        }                                        \
    } while (0)

static cudaError_t run(unsigned int word, int fail_at, unsigned int *out) {
    g_word = word;
    g_reads = g_writes = g_waits = g_calls = 0;
    g_fail_at = fail_at;
    *out = 7;
    return swiglu::fetch_and_clear(g_word, out, nullptr);
}

int main() {
    unsigned int out;
    // a clear word: one read, waited for, and nothing written
    REQUIRE(run(0, 0, &out) == cudaSuccess && out == 0 && g_reads == 1 && g_waits == 1 && g_writes == 0);
    // a set word: handed out and cleared, the write waited for
    REQUIRE(run(1, 0, &out) == cudaSuccess && out == 1 && g_word == 0 && g_writes == 1 && g_waits == 2);
    // an error of any call is the result, and a failed read clears nothing
    for (int i = 1; i <= 4; ++i) REQUIRE(run(1, i, &out) == cudaErrorUnknown && (i > 2 || g_word == 1));
    std::printf("ok 6\n");
    return 0;
}
