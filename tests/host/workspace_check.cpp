// Host-only checks of the table of library-owned workspaces
// (precision_decode_amd/csrc/workspace_table.h), built with g++ and the address
// and undefined-behaviour sanitizers by tests/test_workspace_table.py: growth,
// capture, failed allocations, and host memory that runs out at every
// allocation the table makes.
//
// Prints "workspace_check ok" and exits 0 when every check holds; otherwise
// prints the failed check and exits 1.
#include <cstdint>
#include <cstdio>
#include <cstdlib>
#include <new>

#include "workspace_table.h"

namespace {

int g_failures = 0;
long g_allowed = -1;   // allocations until one fails; negative: none does

#define CHECK(cond)                                                                   \
    do {                                                                              \
        if (!(cond)) {                                                                \
            std::printf("FAILED %s:%d: %s\n", __FILE__, __LINE__, #cond);             \
            ++g_failures;                                                             \
        }                                                                             \
    } while (0)

}  // namespace

void *operator new(size_t n) {
    if (g_allowed == 0) throw std::bad_alloc();
    if (g_allowed > 0) --g_allowed;
    if (void *p = std::malloc(n ? n : 1)) return p;
    throw std::bad_alloc();
}
void operator delete(void *p) noexcept { std::free(p); }
void operator delete(void *p, size_t) noexcept { std::free(p); }

namespace {

void *address(uintptr_t a) { return reinterpret_cast<void *>(a); }

void check_growth() {
    nvfp4ws::WorkspaceTable t;
    uintptr_t next = 0x1000;
    size_t last = 0;
    const auto alloc = [&](size_t bytes) { last = bytes; return address(next += 0x1000); };
    const auto free_run = [] { return false; };
    const auto captured = [] { return true; };
    void *s1 = address(1), *s2 = address(2);
    CHECK(t.get(0, s1, 100, alloc, captured) == nullptr);
    void *a = t.get(0, s1, 100, alloc, free_run);
    CHECK(a && last == 256);
    CHECK(t.get(0, s1, 256, alloc, captured) == a);
    CHECK(t.get(0, s1, 257, alloc, captured) == nullptr);
    void *b = t.get(0, s1, 300, alloc, free_run);
    CHECK(b && b != a && last == 512);
    CHECK(t.get(0, s1, 10, alloc, captured) == b);
    CHECK(t.get(0, s2, 10, alloc, free_run) != b && last == 256);
    CHECK(t.get(1, s1, 10, alloc, free_run) != b);
    CHECK(t.get(0, s1, 5000, [](size_t) -> void * { return nullptr; }, free_run) == nullptr);
    CHECK(t.get(0, s1, 512, alloc, captured) == b);
}

void check_exceptions() {
    for (long allowed = 0; allowed < 4; ++allowed) {
        nvfp4ws::WorkspaceTable t;
        long buffers = 0, got = 0;
        const auto alloc = [&](size_t) { ++buffers; return address(0x1000u * uintptr_t(buffers)); };
        const auto free_run = [] { return false; };
        g_allowed = allowed;
        for (size_t need = 256; need <= 4096; need *= 2) got += t.get(0, nullptr, need, alloc, free_run) != nullptr;
        g_allowed = -1;
        CHECK(got == buffers);   // no buffer is lost
        CHECK(allowed > 0 || got == 0);
        CHECK(t.get(0, nullptr, 1 << 20, alloc, free_run) != nullptr);   // and the table still works
    }
}

}  // namespace

int main() {
    check_growth();
    check_exceptions();
    if (g_failures) return 1;
    std::printf("workspace_check ok\n");
    return 0;
}
