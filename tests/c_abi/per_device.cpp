// A preparation that fails is tried again, and one that has succeeded for a device is not repeated there.
#include "per_device.h"

#include <cstdio>
#include <thread>
#include <vector>

enum Status { kOk = 0, kTransient = 2 };

#define CHECK(x)                                                \
    do {                                                        \
        if (!(x)) {                                             \
            std::printf("line %d: %s\n", __LINE__, #x);         \
            return 1;                                           \
        }                                                       \
    } while (0)

int main()
{
    sdv2::PerDevice once;
    int calls = 0, value = 0;
    auto fails = [&]() { ++calls; return kTransient; };
    auto works = [&]() { ++calls; value = 7; return kOk; };
    CHECK(once.run(3, fails) == kTransient && once.run(3, fails) == kTransient && calls == 2);
    CHECK(once.run(3, works) == kOk && calls == 3 && value == 7);
    CHECK(once.run(3, fails) == kOk && calls == 3);
    CHECK(once.run(0, fails) == kTransient && calls == 4);
    CHECK(once.run(63, works) == kOk && calls == 5);

    for (int turn = 0; turn < 200; ++turn) {       // first calls of several threads: one success, seen by all
        sdv2::PerDevice raced;
        int tries = 0, answer = 0, wrong = 0;
        std::atomic<int> bad{0};
        std::vector<std::thread> threads;
        for (int t = 0; t < 4; ++t)
            threads.emplace_back([&]() {
                while (raced.run(1, [&]() { answer = 5; return ++tries < 3 ? kTransient : kOk; }) != kOk) {}
                if (answer != 5) ++bad;
            });
        for (auto& t : threads) t.join();
        wrong = bad;
        CHECK(wrong == 0 && tries == 3);
    }
    std::printf("ok\n");
    return 0;
}
